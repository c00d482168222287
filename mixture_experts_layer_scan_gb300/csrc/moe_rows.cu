// Rows of tokens in expert order and back, as calls of their own, with their gradients.
//
//   permute             rows[row_of[t][j]] = x[t]                     (zero rows as padding)
//   unpermute           out[t] = sum_j w[t][j] rows[row_of[t][j]]
//   permute, gradient   d_x[t] = sum_j d_rows[row_of[t][j]]           (unpermute without weights)
//   unpermute, gradient d_rows[row_of[t][j]] = w[t][j] d_out[t],  d_w[t][j] = <d_out[t], rows[row_of[t][j]]>
//
// Sums are fp32 in the order of j (the dot products: each lane's columns in order, then a fixed
// butterfly), each result rounded once.  A pair whose row is outside [0, n_rows) has none: it adds nothing
// and its weight's gradient is 0.
//
// All four are bound by HBM: nothing is read twice.  The scatter reads a token's row once for its k stores.
// Rows move as vectors of the widest power of two (16 bytes at most) that divides a row.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {

namespace {

struct RowsDev {
  const void* x;           // scatter: x [T][H]; gather: rows [n_rows][H]
  const void* rows;        // gradient of the gather: rows (nullable)
  const int32_t* row_of;   // [T][k]
  const float* w;          // [T][k] or null
  const int32_t* sorted;   // zero fill: pair of each row (nullable)
  const int32_t* npp;      // rows of the permutation
  void* out;
  float* dw;
  int T, k, n_rows;
  int vpr;                 // vectors per row
  int chunks;              // scatter: runs of 32 * U vectors per row
};

// Rows that hold no pair (sorted[r] >= n_pairs).  A warp looks at up to 32 entries of the list at a time, and at fewer
// where that spreads the rows over more warps (a decode batch over many experts is mostly padding: 64 tokens of
// top-8 over 128 experts in blocks of 16 took 15.4 us with 32).
template <int W>
__device__ __forceinline__ void zero_padding(const RowsDev& p, int unit, int n_units) {
  using V = typename Word<W>::type;
  const int lane = threadIdx.x & 31, npp = min(*p.npp, p.n_rows), n = p.T * p.k;
  const int per = min(32, (npp + n_units - 1) / n_units);
  for (long r0 = (long)unit * per; r0 < npp; r0 += (long)n_units * per) {
    const int r = (int)r0 + lane;
    unsigned pad = __ballot_sync(0xffffffffu, lane < per && r < npp && (unsigned)p.sorted[r] >= (unsigned)n);
    while (pad) {
      const int b = __ffs(pad) - 1;
      pad &= pad - 1;
      V z;
      zero_word(z);
      V* dst = static_cast<V*>(p.out) + (size_t)(r0 + b) * p.vpr;
      for (int v = lane; v < p.vpr; v += 32) dst[v] = z;
    }
  }
}

constexpr int kRowsThreads = 256;
constexpr int kPadCtas = 152;  // CTAs of a launch that fill the padding

// A warp holds U vectors a lane of one token's row and stores them at the rows of its k pairs.
template <int W, int U>
__global__ void __launch_bounds__(kRowsThreads) k_rows_scatter(const RowsDev p) {
  pdl_enter();
  using V = typename Word<W>::type;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int warps = kRowsThreads / 32;
  const int pad_ctas = p.sorted ? kPadCtas : 0;
  if ((int)blockIdx.x < pad_ctas) {
    zero_padding<W>(p, blockIdx.x * warps + warp, pad_ctas * warps);
    return;
  }
  const long units = (long)p.T * p.chunks;
  for (long u = (long)(blockIdx.x - pad_ctas) * warps + warp; u < units; u += (long)(gridDim.x - pad_ctas) * warps) {
    const int t = (int)(u / p.chunks), v0 = (int)(u % p.chunks) * (32 * U) + lane;
    const V* src = static_cast<const V*>(p.x) + (size_t)t * p.vpr;
    V buf[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v0 + 32 * i < p.vpr) buf[i] = src[v0 + 32 * i];
    for (int j0 = 0; j0 < p.k; j0 += 32) {
      const int mine = j0 + lane < p.k ? p.row_of[(size_t)t * p.k + j0 + lane] : -1;
      const int kk = min(32, p.k - j0);
      for (int j = 0; j < kk; ++j) {
        const int r = __shfl_sync(0xffffffffu, mine, j);
        if ((unsigned)r >= (unsigned)p.n_rows) continue;
        V* dst = static_cast<V*>(p.out) + (size_t)r * p.vpr;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (v0 + 32 * i < p.vpr) dst[v0 + 32 * i] = buf[i];
      }
    }
  }
}

// A thread sums one vector of a token over its rows, kGatherRows of them in flight.
constexpr int kGatherRows = 8;
template <typename T, int W>
__global__ void __launch_bounds__(kRowsThreads) k_rows_gather(const RowsDev p) {
  pdl_enter();
  using V = typename Word<W>::type;
  constexpr int N = W / sizeof(T);
  const V* rows = static_cast<const V*>(p.x);
  const int v = blockIdx.y * kRowsThreads + threadIdx.x;
  if (v >= p.vpr) return;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t f0 = (size_t)t * p.k;
    float acc[N] = {};
    for (int j0 = 0; j0 < p.k; j0 += kGatherRows) {
      V u[kGatherRows];
      float wj[kGatherRows];
#pragma unroll
      for (int j = 0; j < kGatherRows; ++j) {
        const int at = j0 + j < p.k ? p.row_of[f0 + j0 + j] : -1;
        const bool in = (unsigned)at < (unsigned)p.n_rows;
        zero_word(u[j]);
        if (in) u[j] = __ldcs(rows + (size_t)at * p.vpr + v);
        wj[j] = !in ? 0.f : p.w ? p.w[f0 + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < kGatherRows; ++j) {
        if (j0 + j >= p.k) break;
        float f[N];
        widen<T, W>(u[j], f);
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = fmaf(wj[j], f[c], acc[c]);
      }
    }
    static_cast<V*>(p.out)[(size_t)t * p.vpr + v] = narrow<T, W>(acc);
  }
}

// Gradient of the weighted sum: a CTA per token, a warp per pair (the pairs' reads of d_out meet in L1).
constexpr int kGradUnroll = 4;
template <typename T, int W>
__global__ void __launch_bounds__(kRowsThreads) k_rows_gather_grad(const RowsDev p) {
  pdl_enter();
  using V = typename Word<W>::type;
  constexpr int N = W / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int pad_ctas = p.sorted ? kPadCtas : 0;
  if ((int)blockIdx.x < pad_ctas) {
    zero_padding<W>(p, blockIdx.x * warps + warp, pad_ctas * warps);
    return;
  }
  for (int t = blockIdx.x - pad_ctas; t < p.T; t += gridDim.x - pad_ctas) {
    const V* d = static_cast<const V*>(p.x) + (size_t)t * p.vpr;
    for (int j = warp; j < p.k; j += warps) {
      const size_t f = (size_t)t * p.k + j;
      const int r = p.row_of[f];
      const bool in = (unsigned)r < (unsigned)p.n_rows;
      if (!in) {
        if (p.dw && lane == 0) p.dw[f] = 0.f;
        continue;
      }
      const float wj = p.w ? p.w[f] : 1.f;
      const V* src = p.dw ? static_cast<const V*>(p.rows) + (size_t)r * p.vpr : nullptr;
      V* dst = p.out ? static_cast<V*>(p.out) + (size_t)r * p.vpr : nullptr;
      float dot = 0.f;
      for (int v0 = lane; v0 < p.vpr; v0 += 32 * kGradUnroll) {
        V a[kGradUnroll], b[kGradUnroll];
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i) {
          const int v = v0 + 32 * i;
          zero_word(a[i]);
          zero_word(b[i]);
          if (v < p.vpr) {
            a[i] = d[v];
            if (src) b[i] = __ldcs(src + v);
          }
        }
#pragma unroll
        for (int i = 0; i < kGradUnroll; ++i) {
          const int v = v0 + 32 * i;
          float fa[N], fb[N];
          widen<T, W>(a[i], fa);
          widen<T, W>(b[i], fb);
#pragma unroll
          for (int c = 0; c < N; ++c) {
            dot = fmaf(fa[c], fb[c], dot);
            fa[c] *= wj;
          }
          if (dst && v < p.vpr) dst[v] = narrow<T, W>(fa);
        }
      }
      if (p.dw) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) p.dw[f] = dot;
      }
    }
  }
}

template <int W>
cudaError_t scatter(RowsDev& p, long row_bytes, cudaStream_t s) {
  p.vpr = (int)(row_bytes / W);
  // few rows: one vector a lane, so that they spread over more warps
  const long units4 = (long)p.T * ((p.vpr + 127) / 128);
  const bool few = units4 < 152 * 16;
  const int per = few ? 32 : 128;
  p.chunks = (p.vpr + per - 1) / per;
  const long units = (long)p.T * p.chunks;
  const int ctas = (int)std::min<long>((units + 7) / 8, 1 << 20) + (p.sorted ? kPadCtas : 0);
  if (few) MOE_LAUNCH((k_rows_scatter<W, 1>), dim3(ctas), dim3(kRowsThreads), 0, s, p);
  else MOE_LAUNCH((k_rows_scatter<W, 4>), dim3(ctas), dim3(kRowsThreads), 0, s, p);
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t gather(RowsDev& p, long row_bytes, cudaStream_t s) {
  p.vpr = (int)(row_bytes / W);
  const int cols = (p.vpr + kRowsThreads - 1) / kRowsThreads;
  if (cols > 65535) return cudaErrorInvalidValue;
  const dim3 grid(std::min(p.T, std::max(1, 152 * 16 / cols)), cols);
  MOE_LAUNCH((k_rows_gather<T, W>), grid, dim3(kRowsThreads), 0, s, p);
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t gather_grad(RowsDev& p, long row_bytes, cudaStream_t s) {
  p.vpr = (int)(row_bytes / W);
  const int warps = std::min(p.k, kRowsThreads / 32);
  const int ctas = std::min(p.T, 1 << 20) + (p.sorted ? kPadCtas : 0);
  MOE_LAUNCH((k_rows_gather_grad<T, W>), dim3(ctas), dim3(32 * warps), 0, s, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_scatter(const void* x, int T, int H, int k, int elem_bytes, const int32_t* row_of,
                                const int32_t* sorted, const int32_t* npp, int n_rows, void* rows, cudaStream_t s) {
  RowsDev p = {};
  p.x = x;
  p.row_of = row_of;
  p.sorted = sorted;
  p.npp = npp;
  p.out = rows;
  p.T = T;
  p.k = k;
  p.n_rows = n_rows;
  const long b = (long)H * elem_bytes;
  switch (row_word(b)) {
    case 16: return scatter<16>(p, b, s);
    case 8: return scatter<8>(p, b, s);
    case 4: return scatter<4>(p, b, s);
    default: return scatter<2>(p, b, s);
  }
}

cudaError_t launch_rows_gather(const void* rows, int n_rows, const int32_t* row_of, const float* w, int T, int H, int k,
                               bool bf16, void* out, cudaStream_t s) {
  RowsDev p = {};
  p.x = rows;
  p.row_of = row_of;
  p.w = w;
  p.out = out;
  p.T = T;
  p.k = k;
  p.n_rows = n_rows;
  const long b = (long)H * (bf16 ? 2 : 4);
  switch (row_word(b)) {
    case 16: return bf16 ? gather<__nv_bfloat16, 16>(p, b, s) : gather<float, 16>(p, b, s);
    case 8: return bf16 ? gather<__nv_bfloat16, 8>(p, b, s) : gather<float, 8>(p, b, s);
    case 4: return bf16 ? gather<__nv_bfloat16, 4>(p, b, s) : gather<float, 4>(p, b, s);
    default: return gather<__nv_bfloat16, 2>(p, b, s);
  }
}

cudaError_t launch_rows_gather_grad(const void* d_out, const void* rows, int n_rows, const int32_t* row_of,
                                    const float* w, const int32_t* sorted, const int32_t* npp, int T, int H, int k,
                                    bool bf16, void* d_rows, float* d_w, cudaStream_t s) {
  RowsDev p = {};
  p.x = d_out;
  p.rows = rows;
  p.row_of = row_of;
  p.w = w;
  p.sorted = d_rows ? sorted : nullptr;
  p.npp = npp;
  p.out = d_rows;
  p.dw = d_w;
  p.T = T;
  p.k = k;
  p.n_rows = n_rows;
  const long b = (long)H * (bf16 ? 2 : 4);
  switch (row_word(b)) {
    case 16: return bf16 ? gather_grad<__nv_bfloat16, 16>(p, b, s) : gather_grad<float, 16>(p, b, s);
    case 8: return bf16 ? gather_grad<__nv_bfloat16, 8>(p, b, s) : gather_grad<float, 8>(p, b, s);
    case 4: return bf16 ? gather_grad<__nv_bfloat16, 4>(p, b, s) : gather_grad<float, 4>(p, b, s);
    default: return gather_grad<__nv_bfloat16, 2>(p, b, s);
  }
}

}  // namespace moe
