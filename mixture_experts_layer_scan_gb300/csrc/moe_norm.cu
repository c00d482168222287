// Norms before and after a block, with the block's gate and residual scale, and their gradients.
//
//   prenorm    h = x r w,  r = (mean x^2 + eps)^-1/2
//   postnorm   n = y r_y,  v = n post_w (v = y without a norm),  out = res_scale x + scale G v,
//              h = out r_o next_w (the next block's prenorm, from the unrounded out)
//   gradients  of a norm n = x r with d_n = g:  d_x = r (g - n mean(g n))
//              D = d_out + that of h at out;  d_x = res_scale D,  d_v = scale G D,  d_G = scale D v,
//              d_post_w = sum_t d_v n,  d_next_w = sum_t d_h out r_o,  d_y from d_v post_w
//
// Everything is fp32 between the loads and the one rounding of each result.  The gradients recompute the
// forward pass from x and y: statistics kept by the forward pass would save no bytes, and a rounded out
// would not be the one that the norm saw.
//
// Bound by HBM: a CTA takes a row, every element is read once and stays in registers across the sums
// over the row.  The weights' gradients are sums over rows: a CTA keeps those of its rows in registers,
// writes one fp32 row of partial sums, and a second kernel adds the CTAs' rows in their order.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {

namespace {

// N consecutive values of a weight (or gate) vector of fp32 or bf16
template <int N>
__device__ __forceinline__ void load_w(const void* w, bool f32, size_t i, float (&f)[N]) {
  constexpr int WB = N * 2;  // bytes of N bf16
  if (f32) {
    constexpr int WF = N * 4 >= 16 ? 16 : N * 4;
    using V = typename Word<WF>::type;
    constexpr int per = WF / 4;
#pragma unroll
    for (int q = 0; q < N / per; ++q) {
      float g[per];
      widen<float, WF>(reinterpret_cast<const V*>(static_cast<const float*>(w) + i)[q], g);
#pragma unroll
      for (int c = 0; c < per; ++c) f[q * per + c] = g[c];
    }
  } else {
    using V = typename Word<WB>::type;
    widen<__nv_bfloat16, WB>(*reinterpret_cast<const V*>(static_cast<const uint16_t*>(w) + i), f);
  }
}

__device__ __forceinline__ float load_one(const void* w, bool f32, size_t i) {
  return f32 ? static_cast<const float*>(w)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(w)[i]);
}

// bf16 rows take the approximate exponential and quotient (off by some 2^-21, far below a step of theirs): with the
// rounded ones a full gate of 16384 x 4096 was bound by their instructions.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-z));
  return 1.0f / (1.0f + expf(-z));
}

// Sums of two values over the CTA, in every thread (fixed order).  `s` is not reused before a barrier.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return make_float2(a, b);
  if (lane == 0) s[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 v = lane < warps ? s[lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

struct NormDev {
  const void *x, *y, *post_w, *gate, *next_w;
  const void *d_out, *d_h;
  void *out, *h;
  void *d_x, *d_y, *d_gate;
  float* part;       // partial sums: [3][gridDim.x][H] of d_post_w, d_next_w, d_gate
  int T, H;
  float inv_h, eps, scale, res_scale;
  int gate_kind;     // MOE_GATE_*
  bool sigmoid, w_f32, gate_f32;
  bool sum_post, sum_next, sum_gate;
};

// The gate of N elements of row t (1 without a gate).
template <typename T, int N>
__device__ __forceinline__ void load_gate(const NormDev& p, int t, int i, float token, float (&g)[N]) {
  if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
    load_w<N>(p.gate, p.gate_f32, (p.gate_kind == MOE_GATE_FULL ? (size_t)t * p.H : 0) + i, g);
    if (p.sigmoid) {
#pragma unroll
      for (int c = 0; c < N; ++c) g[c] = sigmoid<T>(g[c]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) g[c] = token;
  }
}
template <typename T>
__device__ __forceinline__ float token_gate(const NormDev& p, int t) {
  if (p.gate_kind != MOE_GATE_TOKEN) return 1.0f;
  const float g = load_one(p.gate, p.gate_f32, t);
  return p.sigmoid ? sigmoid<T>(g) : g;
}

// Persistent: a CTA takes every gridDim-th row and holds the next one's loads while it is at work on this one.
// Thread i holds vectors i, i + blockDim, ... (NV of them).  The sums' shared memory alternates from row to row: what a
// row wrote is overwritten two barriers later.  Measured, 16384 x 4096 bf16 with a token gate (us): a CTA to a row
// with 8 elements a thread 164, with 16 107.
template <typename T, int W, int NV, bool POST>
__global__ void __launch_bounds__(512) k_norm(const NormDev p) {
  pdl_enter();
  using V = typename Word<W>::type;
  constexpr int N = W / sizeof(T);
  __shared__ float2 sums[2][2][32];
  const int vpr = p.H / N;
  V xv[NV], yv[POST ? NV : 1];
  auto fetch = [&](int t) {
    const V* xr = reinterpret_cast<const V*>(static_cast<const T*>(p.x) + (size_t)t * p.H);
    const V* yr = reinterpret_cast<const V*>(static_cast<const T*>(p.y) + (size_t)t * p.H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < vpr) {
        xv[i] = xr[v];
        if constexpr (POST) yv[i] = yr[v];
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    zero_word(xv[i]);
    if constexpr (POST) zero_word(yv[i]);
  }
  if ((int)blockIdx.x < p.T) fetch(blockIdx.x);
  int par = 0;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    float o[NV][N], y[POST ? NV : 1][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      widen<T, W>(xv[i], o[i]);
      if constexpr (POST) widen<T, W>(yv[i], y[i]);
    }
    if (t + (int)gridDim.x < p.T) fetch(t + gridDim.x);
    if constexpr (POST) {
      float ry = 1.0f;
      if (p.post_w) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int c = 0; c < N; ++c) a = fmaf(y[i][c], y[i][c], a);
        ry = rsqrtf(block_sum2(a, 0.f, sums[par][0]).x * p.inv_h + p.eps);
      }
      const float tok = p.scale * token_gate<T>(p, t);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vpr) break;
        float g[N];
        if (p.post_w) {
          float w[N];
          load_w<N>(p.post_w, p.w_f32, (size_t)v * N, w);
#pragma unroll
          for (int c = 0; c < N; ++c) y[i][c] *= ry * w[c];
        }
        if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
          load_gate<T, N>(p, t, v * N, 1.0f, g);
#pragma unroll
          for (int c = 0; c < N; ++c) y[i][c] *= g[c];
        }
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] = fmaf(p.res_scale, o[i][c], tok * y[i][c]);
        reinterpret_cast<V*>(static_cast<T*>(p.out) + (size_t)t * p.H)[v] = narrow<T, W>(o[i]);
      }
    }
    if (!POST || p.next_w) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int c = 0; c < N; ++c) a = fmaf(o[i][c], o[i][c], a);
      }
      const float r = rsqrtf(block_sum2(a, 0.f, sums[par][1]).x * p.inv_h + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vpr) break;
        float w[N];
        load_w<N>(p.next_w, p.w_f32, (size_t)v * N, w);
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] *= r * w[c];
        reinterpret_cast<V*>(static_cast<T*>(p.h) + (size_t)t * p.H)[v] = narrow<T, W>(o[i]);
      }
    }
  }
}

// Gradients; the prenorm's is POST = false with x in the place of out and d_out = 0.
template <typename T, int W, int NV, bool POST>
__global__ void __launch_bounds__(NV * (W / (int)sizeof(T)) > 8 ? 1024 : 512) k_norm_grad(const NormDev p) {
  pdl_enter();
  using V = typename Word<W>::type;
  constexpr int N = W / sizeof(T);
  __shared__ float2 s1[32], s2[32], s3[32];
  const int vpr = p.H / N;
  float acc_n[NV][N] = {}, acc_p[POST ? NV : 1][N] = {}, acc_g[POST ? NV : 1][N] = {};
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t at = (size_t)t * p.H;
    V xv[NV], dhv[NV], yv[POST ? NV : 1], dov[POST ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      zero_word(xv[i]);
      zero_word(dhv[i]);
      if constexpr (POST) {
        zero_word(yv[i]);
        zero_word(dov[i]);
      }
      if (v < vpr) {
        xv[i] = reinterpret_cast<const V*>(static_cast<const T*>(p.x) + at)[v];
        if (p.d_h) dhv[i] = reinterpret_cast<const V*>(static_cast<const T*>(p.d_h) + at)[v];
        if constexpr (POST) {
          yv[i] = reinterpret_cast<const V*>(static_cast<const T*>(p.y) + at)[v];
          if (p.d_out) dov[i] = reinterpret_cast<const V*>(static_cast<const T*>(p.d_out) + at)[v];
        }
      }
    }
    float o[NV][N], n[POST ? NV : 1][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) widen<T, W>(xv[i], o[i]);
    float ry = 1.0f, tok = 1.0f;
    if constexpr (POST) {
      if (p.post_w) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float y[N];
          widen<T, W>(yv[i], y);
#pragma unroll
          for (int c = 0; c < N; ++c) a = fmaf(y[c], y[c], a);
        }
        ry = rsqrtf(block_sum2(a, 0.f, s1).x * p.inv_h + p.eps);
      }
      tok = token_gate<T>(p, t);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        widen<T, W>(yv[i], n[i]);
#pragma unroll
        for (int c = 0; c < N; ++c) n[i][c] *= ry;
        if (v >= vpr) continue;
        float w[N], g[N];
#pragma unroll
        for (int c = 0; c < N; ++c) w[c] = 1.f;
        if (p.post_w) load_w<N>(p.post_w, p.w_f32, (size_t)v * N, w);
        load_gate<T, N>(p, t, v * N, tok, g);
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] = fmaf(p.res_scale, o[i][c], p.scale * g[c] * (n[i][c] * w[c]));
      }
    }
    // D, in place of d_out
    float D[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (POST) {
        widen<T, W>(dov[i], D[i]);
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c) D[i][c] = 0.f;
      }
    }
    if (p.d_h) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vpr) break;
        float d[N], w[N];
        widen<T, W>(dhv[i], d);
        load_w<N>(p.next_w, p.w_f32, (size_t)v * N, w);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          a = fmaf(o[i][c], o[i][c], a);
          b = fmaf(o[i][c], d[c] * w[c], b);
        }
      }
      const float2 s = block_sum2(a, b, s2);
      const float r = rsqrtf(s.x * p.inv_h + p.eps);
      const float m = s.y * r * p.inv_h;  // mean(g n)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vpr) break;
        float d[N], w[N];
        widen<T, W>(dhv[i], d);
        load_w<N>(p.next_w, p.w_f32, (size_t)v * N, w);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float nn = o[i][c] * r;
          acc_n[i][c] = fmaf(d[c], nn, acc_n[i][c]);
          D[i][c] += r * (d[c] * w[c] - nn * m);
        }
      }
    }
    if constexpr (!POST) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < vpr) reinterpret_cast<V*>(static_cast<T*>(p.d_x) + at)[v] = narrow<T, W>(D[i]);
      }
    } else {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vpr) break;
        float dx[N], w[N], g[N], dg[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
          dx[c] = p.res_scale * D[i][c];
          w[c] = 1.f;
        }
        reinterpret_cast<V*>(static_cast<T*>(p.d_x) + at)[v] = narrow<T, W>(dx);
        if (p.post_w) load_w<N>(p.post_w, p.w_f32, (size_t)v * N, w);
        load_gate<T, N>(p, t, v * N, tok, g);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float z = p.scale * D[i][c];
          dg[c] = z * (n[i][c] * w[c]);
          if (p.sigmoid) dg[c] *= g[c] * (1.0f - g[c]);
          const float dv = z * g[c];
          acc_p[i][c] = fmaf(dv, n[i][c], acc_p[i][c]);
          acc_g[i][c] += dg[c];
          b += dg[c];
          D[i][c] = dv * w[c];  // from here on the gradient in n
          a = fmaf(D[i][c], n[i][c], a);
        }
        if (p.gate_kind == MOE_GATE_FULL && p.d_gate) {
          if (p.gate_f32) {
#pragma unroll
            for (int c = 0; c < N; ++c) static_cast<float*>(p.d_gate)[at + (size_t)v * N + c] = dg[c];
          } else {
            using G = typename Word<N * 2>::type;
            reinterpret_cast<G*>(static_cast<uint16_t*>(p.d_gate) + at)[v] = narrow<__nv_bfloat16, N * 2>(dg);
          }
        }
      }
      float m = 0.f;
      if (p.post_w || p.gate_kind == MOE_GATE_TOKEN) {
        const float2 s = block_sum2(a, b, s3);
        m = p.post_w ? s.x * p.inv_h : 0.f;
        if (p.gate_kind == MOE_GATE_TOKEN && p.d_gate && threadIdx.x == 0) static_cast<float*>(p.d_gate)[t] = s.y;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vpr) break;
        float dy[N];
#pragma unroll
        for (int c = 0; c < N; ++c) dy[c] = p.post_w ? ry * (D[i][c] - n[i][c] * m) : D[i][c];
        reinterpret_cast<V*>(static_cast<T*>(p.d_y) + at)[v] = narrow<T, W>(dy);
      }
    }
    if (t + (int)gridDim.x < p.T) __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= vpr) break;
    float* row = p.part + (size_t)blockIdx.x * p.H + (size_t)v * N;
    const size_t plane = (size_t)gridDim.x * p.H;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (p.sum_next) row[plane + c] = acc_n[i][c];
      if constexpr (POST) {
        if (p.sum_post) row[c] = acc_p[i][c];
        if (p.sum_gate) row[2 * plane + c] = acc_g[i][c];
      }
    }
  }
}

// out[z][c] = sum_g part[z][g][c], 32 columns to a CTA, its 8 warps' runs of rows added in their order
struct SumDev {
  const float* part;
  float* out[3];
  int rows, H;
};
__global__ void __launch_bounds__(256) k_sum_rows(const SumDev p) {
  pdl_enter();
  __shared__ float s[8][32];
  float* out = p.out[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* part = p.part + (size_t)blockIdx.y * p.rows * p.H + c;
  const int per = (p.rows + 7) / 8, g0 = min(p.rows, warp * per), g1 = min(p.rows, g0 + per);
  float a = 0.f;
  if (c < p.H) {
#pragma unroll 8
    for (int g = g0; g < g1; ++g) a += part[(size_t)g * p.H];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < p.H) {
    a = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) a += s[w][lane];
    out[c] = a;
  }
}

// Elements of a thread of the gradients: 8, or 16 for rows that 512 threads do not hold with 8.
int threads_for(int H, int per) { return std::max(32, ((H + per - 1) / per + 31) / 32 * 32); }
bool wide_row(int H) { return H > 8 * 512; }

// CTAs of a forward kernel that are resident together
template <typename T, int W, int NV, bool POST>
int resident(int threads) {
  static int known[64][17] = {};  // (by device and warps; racing threads write the same)
  int dev = 0;
  cudaGetDevice(&dev);
  int* at = dev >= 0 && dev < 64 && threads <= 512 ? &known[dev][threads / 32] : nullptr;
  if (at && *at) return *at;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_norm<T, W, NV, POST>, threads, 0) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  if (at) *at = n * 152;
  return n * 152;
}

template <typename T, int W, int NV, bool POST>
cudaError_t launch_forward(const NormDev& p, cudaStream_t s) {
  const int threads = threads_for(p.H, NV * (W / (int)sizeof(T)));
  const int grid = std::min(p.T, resident<T, W, NV, POST>(threads));
  MOE_LAUNCH((k_norm<T, W, NV, POST>), dim3(grid), dim3(threads), 0, s, p);
  return cudaGetLastError();
}

template <typename T, int W, int NV, bool POST>
cudaError_t launch_gradient(const NormDev& p, int grid, cudaStream_t s) {
  MOE_LAUNCH((k_norm_grad<T, W, NV, POST>), dim3(grid), dim3(threads_for(p.H, NV * (W / (int)sizeof(T)))), 0, s, p);
  return cudaGetLastError();
}

template <typename T, int W, bool POST>
cudaError_t launch_width(const NormDev& p, bool grad, int grid, cudaStream_t s) {
  constexpr int N = W / sizeof(T);
  if (grad) return wide_row(p.H) ? launch_gradient<T, W, 16 / N, POST>(p, grid, s) : launch_gradient<T, W, 8 / N, POST>(p, grid, s);
  // elements of a thread: 16; few rows 8 (a row is over sooner: one of 4096 1.6 us instead of 1.8); long ones 32
  if (p.H > 512 * 16) return launch_forward<T, W, 32 / N, POST>(p, s);
  if (p.T <= 304 && p.H <= 512 * 8) return launch_forward<T, W, 8 / N, POST>(p, s);
  return launch_forward<T, W, 16 / N, POST>(p, s);
}
template <typename T, int W>
cudaError_t launch_width(const NormDev& p, bool post, bool grad, int grid, cudaStream_t s) {
  return post ? launch_width<T, W, true>(p, grad, grid, s) : launch_width<T, W, false>(p, grad, grid, s);
}

cudaError_t launch_typed(const NormDev& p, bool bf16, bool post, bool grad, int grid, cudaStream_t s) {
  const int w = row_word((long)p.H * (bf16 ? 2 : 4));
  if (bf16)
    return w == 16  ? launch_width<__nv_bfloat16, 16>(p, post, grad, grid, s)
           : w >= 4 ? launch_width<__nv_bfloat16, 4>(p, post, grad, grid, s)
                    : launch_width<__nv_bfloat16, 2>(p, post, grad, grid, s);
  return w == 16 ? launch_width<float, 16>(p, post, grad, grid, s) : launch_width<float, 4>(p, post, grad, grid, s);
}

NormDev make_dev(const NormArgs& a) {
  NormDev p = {};
  p.x = a.x;
  p.y = a.y;
  p.post_w = a.post_w;
  p.gate = a.gate;
  p.next_w = a.next_w;
  p.d_out = a.d_out;
  p.d_h = a.d_h;
  p.out = a.out;
  p.h = a.h;
  p.d_x = a.d_x;
  p.d_y = a.d_y;
  p.d_gate = a.d_gate;
  p.T = a.T;
  p.H = a.H;
  p.inv_h = 1.0f / (float)a.H;
  p.eps = a.rule.eps;
  p.scale = a.rule.scale;
  p.res_scale = a.rule.res_scale;
  p.gate_kind = a.rule.gate;
  p.sigmoid = a.rule.gate_sigmoid != 0 && a.rule.gate != MOE_GATE_NONE;
  p.w_f32 = a.rule.w_dtype == MOE_F32;
  p.gate_f32 = a.rule.gate_dtype == MOE_F32;
  return p;
}

}  // namespace

int norm_grad_rows(int T, int H) { return std::min(T, 152 * std::max(1, 512 / threads_for(H, wide_row(H) ? 16 : 8))); }

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  const NormDev p = make_dev(a);
  return launch_typed(p, a.bf16, a.y != nullptr, false, 0, s);
}

cudaError_t launch_norm_grad(const NormArgs& a, cudaStream_t s) {
  NormDev p = make_dev(a);
  const bool channel = a.rule.gate == MOE_GATE_CHANNEL;
  p.part = static_cast<float*>(a.workspace);
  p.sum_post = a.d_post_w != nullptr;
  p.sum_next = a.d_next_w != nullptr;
  p.sum_gate = channel && a.d_gate;
  const int rows = norm_grad_rows(a.T, a.H);
  const cudaError_t e = launch_typed(p, a.bf16, a.y != nullptr, true, rows, s);
  if (e != cudaSuccess || !(p.sum_post || p.sum_next || p.sum_gate)) return e;
  SumDev q = {};
  q.part = p.part;
  q.out[0] = a.d_post_w;
  q.out[1] = a.d_next_w;
  q.out[2] = p.sum_gate ? static_cast<float*>(a.d_gate) : nullptr;
  q.rows = rows;
  q.H = a.H;
  MOE_LAUNCH(k_sum_rows, dim3((a.H + 31) / 32, 3), dim3(256), 0, s, q);
  return cudaGetLastError();
}

}  // namespace moe
