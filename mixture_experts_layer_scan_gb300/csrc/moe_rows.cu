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
// All four are bound by HBM: nothing is read twice from there.  The scatter reads a token's row once for its k stores.
// Rows of whole 16-byte units move as those.  Other rows begin anywhere: there a thread takes an aligned unit of the row
// that is written, puts the other row's bytes for it together from the two units that hold them, and goes by
// elements only at the row's ends (by elements throughout, 9218 x 3 rows of 2475 bf16 took 131 us to sum).
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
  int vpr;                 // 16-byte vectors per row
  int chunks;              // scatter: runs of 32 * U vectors per row
  int pad_ctas;            // the launch's first CTAs, which fill the padding
};

constexpr int kRowsThreads = 256;
// CTAs that fill the padding: a warp to each row that may be padding, from 8 warps of an SM on to 32.  (A few tokens
// over many experts are mostly padding: 200 x 3 rows of 2968 fp32 over 256 experts in blocks of 64, with 456 warps, took
// 70 us.)
int pad_ctas(const RowsDev& p, int threads) {
  if (!p.sorted) return 0;
  const long rows = std::max(0l, (long)p.n_rows - (long)p.T * p.k), warps = threads / 32;
  return (int)((std::min(std::max(rows, 152l * 8), 152l * 32) + warps - 1) / warps);
}

// Rows that hold no pair (sorted[r] >= n_pairs).  A warp looks at up to 32 entries of the list at a time, and at fewer
// where that spreads the rows over more warps (a decode batch over many experts is mostly padding: 64 tokens of
// top-8 over 128 experts in blocks of 16 took 15.4 us with 32).
template <typename Zero>
__device__ __forceinline__ void zero_padding(const RowsDev& p, int unit, int n_units, Zero zero) {
  const int lane = threadIdx.x & 31, npp = min(*p.npp, p.n_rows), n = p.T * p.k;
  const int per = min(32, (npp + n_units - 1) / n_units);
  for (long r0 = (long)unit * per; r0 < npp; r0 += (long)n_units * per) {
    const int r = (int)r0 + lane;
    unsigned pad = __ballot_sync(0xffffffffu, lane < per && r < npp && (unsigned)p.sorted[r] >= (unsigned)n);
    while (pad) {
      const int b = __ffs(pad) - 1;
      pad &= pad - 1;
      zero((size_t)(r0 + b));
    }
  }
}
// The padding's share of a launch's first CTAs, rows of whole units.
__device__ __forceinline__ bool pad_cta(const RowsDev& p) {
  const int ctas = p.pad_ctas, warps = blockDim.x >> 5;
  if ((int)blockIdx.x >= ctas) return false;
  zero_padding(p, blockIdx.x * warps + (threadIdx.x >> 5), ctas * warps, [&](size_t row) {
    uint4* dst = static_cast<uint4*>(p.out) + row * p.vpr;
    for (int v = threadIdx.x & 31; v < p.vpr; v += 32) dst[v] = make_uint4(0, 0, 0, 0);
  });
  return true;
}

// A warp holds U vectors a lane of one token's row and stores them at the rows of its k pairs: 8192 tokens of 8 pairs of
// 4096 bf16 97 us, 6.2 TB/s, 92 % of a copy's rate (nine tenths of the bytes are writes).
template <int U>
__global__ void __launch_bounds__(kRowsThreads) k_rows_scatter(const RowsDev p) {
  pdl_enter();
  using V = uint4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int warps = kRowsThreads / 32;
  if (pad_cta(p)) return;
  const long units = (long)p.T * p.chunks;
  for (long u = (long)(blockIdx.x - p.pad_ctas) * warps + warp; u < units; u += (long)(gridDim.x - p.pad_ctas) * warps) {
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

// A thread sums one vector of a token over its rows, kGatherRows of them in flight (4099 tokens of 6 rows of 2048 fp32:
// 32.5 us, 7.2 TB/s, as some of the output stays in L2).
constexpr int kGatherRows = 8;
template <typename T>
__global__ void __launch_bounds__(kRowsThreads) k_rows_gather(const RowsDev p) {
  pdl_enter();
  using V = uint4;
  constexpr int N = 16 / sizeof(T);
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
        widen<T, 16>(u[j], f);
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = fmaf(wj[j], f[c], acc[c]);
      }
    }
    static_cast<V*>(p.out)[(size_t)t * p.vpr + v] = narrow<T, 16>(acc);
  }
}

// Gradient of the weighted sum: a CTA per token, a warp per pair (the pairs' reads of d_out meet in L1).  8192 tokens of
// 8 rows of 4096 bf16: 174 us, 6.5 TB/s, 97 % of a copy's rate.
// WIDE, for few pairs: a CTA per pair (a warp's way through a long row is a chain of memory's latencies: 56 x 8 rows of
// 5185 fp32 took 50 us).
constexpr int kGradUnroll = 4;
constexpr long kWidePairs = 152 * 8;   // at most
constexpr long kWideBytes = 4096;      // of a row at least

// The pairs of a CTA, pair(t, j); then the sum of a pair's products over its warp or CTA, in a fixed order.
template <bool WIDE, typename F>
__device__ __forceinline__ void each_pair(const RowsDev& p, F pair) {
  const long at = blockIdx.x - p.pad_ctas, step = gridDim.x - p.pad_ctas;
  if constexpr (WIDE) {
    for (long f = at; f < (long)p.T * p.k; f += step) pair((int)(f / p.k), (int)(f % p.k));
  } else {
    for (long t = at; t < p.T; t += step)
      for (int j = threadIdx.x >> 5; j < p.k; j += blockDim.x >> 5) pair((int)t, j);
  }
}
template <bool WIDE>
__device__ __forceinline__ float pair_sum(float dot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if constexpr (WIDE) {
    __shared__ float s[kRowsThreads / 32];
    __syncthreads();  // (the pair before has been read)
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = dot;
    __syncthreads();
    dot = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsThreads / 32; ++w) dot += s[w];
  }
  return dot;
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowsThreads) k_rows_gather_grad(const RowsDev p) {
  pdl_enter();
  using V = uint4;
  constexpr int N = 16 / sizeof(T);
  if (pad_cta(p)) return;
  const int me = WIDE ? threadIdx.x : threadIdx.x & 31, team = WIDE ? kRowsThreads : 32;
  each_pair<WIDE>(p, [&](int t, int j) {
    const V* d = static_cast<const V*>(p.x) + (size_t)t * p.vpr;
    const size_t f = (size_t)t * p.k + j;
    const int r = p.row_of[f];
    const bool in = (unsigned)r < (unsigned)p.n_rows;
    if (!in) {
      if (p.dw && me == 0) p.dw[f] = 0.f;
      return;
    }
    const float wj = p.w ? p.w[f] : 1.f;
    const V* src = p.dw ? static_cast<const V*>(p.rows) + (size_t)r * p.vpr : nullptr;
    V* dst = p.out ? static_cast<V*>(p.out) + (size_t)r * p.vpr : nullptr;
    float dot = 0.f;
    for (int v0 = me; v0 < p.vpr; v0 += team * kGradUnroll) {
      V a[kGradUnroll], b[kGradUnroll];
#pragma unroll
      for (int i = 0; i < kGradUnroll; ++i) {
        const int v = v0 + team * i;
        zero_word(a[i]);
        zero_word(b[i]);
        if (v < p.vpr) {
          a[i] = d[v];
          if (src) b[i] = __ldcs(src + v);
        }
      }
#pragma unroll
      for (int i = 0; i < kGradUnroll; ++i) {
        const int v = v0 + team * i;
        float fa[N], fb[N];
        widen<T, 16>(a[i], fa);
        widen<T, 16>(b[i], fb);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          dot = fmaf(fa[c], fb[c], dot);
          fa[c] *= wj;
        }
        if (dst && v < p.vpr) dst[v] = narrow<T, 16>(fa);
      }
    }
    if (p.dw) {
      dot = pair_sum<WIDE>(dot);
      if (me == 0) p.dw[f] = dot;
    }
  });
}

// ---- rows that are no whole 16-byte units --------------------------------------------------------------
// The aligned units of a row of a tensor: byte of the first, their number, bytes of the first before the row.
struct Units {
  int n, lead, bytes;
  __device__ __forceinline__ Units(size_t row, size_t row_bytes) : lead((int)((row * row_bytes) & 15)), bytes((int)row_bytes) {
    n = (lead + bytes + 15) / 16;
  }
  __device__ __forceinline__ int from(int u) const { return u * 16 - lead; }  // byte of the row at which unit u begins
  __device__ __forceinline__ bool whole(int u) const { return from(u) >= 0 && from(u) + 16 <= bytes; }
};

// Another row's bytes in the units of a row: unit u is 16 bytes from `at` + 16 u on, `sh` bytes further.
// near_end: some of what those units hold lies outside the tensor, and units are put together by elements.
template <int E>
struct Source {
  const uint8_t *row, *at;
  uint32_t sh;
  bool near_end;
  __device__ __forceinline__ Source(const void* tensor, size_t rows, size_t r, const Units& q) {
    const uint8_t* begin = static_cast<const uint8_t*>(tensor);
    row = begin + r * (size_t)q.bytes;
    const size_t off = r * (size_t)q.bytes + 16;  // (of unit 0, 16 bytes further: not negative)
    const size_t unit = off - q.lead;
    sh = (uint32_t)(unit & 15);
    at = begin + (unit - sh) - 16;
    near_end = unit - sh < 16 || unit - sh - 16 + 16 * (size_t)(q.n + 1) > rows * (size_t)q.bytes;
  }
  // Unit u; what lies outside the row is anything (0 near the tensor's ends).
  __device__ __forceinline__ uint4 load(const Units& q, int u) const {
    if (near_end) return by_elements(q, u);
    const uint4* from = reinterpret_cast<const uint4*>(at) + u;
    const uint4 a = __ldg(from);
    if (sh == 0) return a;
    const uint4 b = __ldg(from + 1);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (sh & 4)
#pragma unroll
      for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
    if (sh & 8)
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
    if (E == 2 && (sh & 2))
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __noinline__ uint4 by_elements(const Units& q, int u) const {
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < 16 / E; ++i) {
      const int b = q.from(u) + i * E;
      if (b < 0 || b >= q.bytes) continue;
      const uint32_t v = *reinterpret_cast<const typename Word<E>::type*>(row + b);
      const int k = i * E / 4;
      const uint32_t bits = E == 2 ? v << (16 * (i & 1)) : v;
      if (k == 0) w[0] |= bits;
      else if (k == 1) w[1] |= bits;
      else if (k == 2) w[2] |= bits;
      else w[3] |= bits;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int E>
__device__ __forceinline__ void store_unit(uint8_t* row, const Units& q, int u, const uint4& v) {
  if (q.whole(u)) {
    *reinterpret_cast<uint4*>(row + q.from(u)) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 16 / E; ++i) {
    const int b = q.from(u) + i * E;
    if (b < 0 || b >= q.bytes) continue;
    *reinterpret_cast<typename Word<E>::type*>(row + b) =
        (typename Word<E>::type)(E == 2 ? w[i / 2] >> (16 * (i & 1)) : w[i]);
  }
}

template <int E>
__device__ __forceinline__ bool pad_cta_odd(const RowsDev& p, size_t row_bytes) {
  const int ctas = p.pad_ctas, warps = blockDim.x >> 5;
  if ((int)blockIdx.x >= ctas) return false;
  zero_padding(p, blockIdx.x * warps + (threadIdx.x >> 5), ctas * warps, [&](size_t row) {
    const Units q(row, row_bytes);
    uint8_t* dst = static_cast<uint8_t*>(p.out) + row * row_bytes;
    for (int u = threadIdx.x & 31; u < q.n; u += 32) store_unit<E>(dst, q, u, make_uint4(0, 0, 0, 0));
  });
  return true;
}

// A warp to a pair (units differ from row to row, so a token's are not held); P > 1, for rows of one unit a lane: P pairs in
// flight (65694 pairs of 109 fp32 with the sort: 36 us with one).
constexpr long kShortBytes = 480;  // 31 units at most
template <int E, int P>
__global__ void __launch_bounds__(kRowsThreads) k_rows_scatter_odd(const RowsDev p, size_t row_bytes) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int warps = kRowsThreads / 32;
  if (pad_cta_odd<E>(p, row_bytes)) return;
  const long pairs = (long)p.T * p.k;
  if constexpr (P > 1) {
    const long step = (long)(gridDim.x - p.pad_ctas) * warps * P;
    for (long f = ((long)(blockIdx.x - p.pad_ctas) * warps + warp) * P; f < pairs; f += step) {
      int r[P];
      uint4 v[P];
#pragma unroll
      for (int i = 0; i < P; ++i) r[i] = f + i < pairs ? p.row_of[f + i] : -1;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if ((unsigned)r[i] >= (unsigned)p.n_rows) continue;
        const Units q(r[i], row_bytes);
        if (lane < q.n) v[i] = Source<E>(p.x, p.T, (f + i) / p.k, q).load(q, lane);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if ((unsigned)r[i] >= (unsigned)p.n_rows) continue;
        const Units q(r[i], row_bytes);
        if (lane < q.n) store_unit<E>(static_cast<uint8_t*>(p.out) + (size_t)r[i] * row_bytes, q, lane, v[i]);
      }
    }
    return;
  }
  for (long f = (long)(blockIdx.x - p.pad_ctas) * warps + warp; f < pairs; f += (long)(gridDim.x - p.pad_ctas) * warps) {
    const int r = p.row_of[f];
    if ((unsigned)r >= (unsigned)p.n_rows) continue;
    const Units q(r, row_bytes);
    const Source<E> src(p.x, p.T, f / p.k, q);
    uint8_t* dst = static_cast<uint8_t*>(p.out) + (size_t)r * row_bytes;
    for (int u0 = lane; u0 < q.n; u0 += 32 * 4) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (u0 + 32 * i < q.n) v[i] = src.load(q, u0 + 32 * i);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (u0 + 32 * i < q.n) store_unit<E>(dst, q, u0 + 32 * i, v[i]);
    }
  }
}

// A thread sums one unit of a token over its rows, four of them in flight.
template <typename T>
__global__ void __launch_bounds__(kRowsThreads) k_rows_gather_odd(const RowsDev p, size_t row_bytes) {
  pdl_enter();
  constexpr int N = 16 / sizeof(T), kFlight = 4;
  const int u = blockIdx.y * blockDim.x + threadIdx.x;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const Units q(t, row_bytes);
    if (u >= q.n) continue;
    const size_t f0 = (size_t)t * p.k;
    float acc[N] = {};
    for (int j0 = 0; j0 < p.k; j0 += kFlight) {
      uint4 y[kFlight];
      float w[kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int at = j0 + j < p.k ? p.row_of[f0 + j0 + j] : -1;
        const bool in = (unsigned)at < (unsigned)p.n_rows;
        w[j] = !in ? 0.f : p.w ? p.w[f0 + j0 + j] : 1.f;
        y[j] = make_uint4(0, 0, 0, 0);
        if (in) y[j] = Source<sizeof(T)>(p.x, p.n_rows, at, q).load(q, u);
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        if (j0 + j >= p.k) break;
        float f[N];
        widen<T, 16>(y[j], f);
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = fmaf(w[j], f[c], acc[c]);
      }
    }
    store_unit<sizeof(T)>(static_cast<uint8_t*>(p.out) + (size_t)t * row_bytes, q, u, narrow<T, 16>(acc));
  }
}

// Pairs as k_rows_gather_grad's.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowsThreads) k_rows_gather_grad_odd(const RowsDev p, size_t row_bytes) {
  pdl_enter();
  constexpr int N = 16 / sizeof(T);
  if (pad_cta_odd<sizeof(T)>(p, row_bytes)) return;
  const int me = WIDE ? threadIdx.x : threadIdx.x & 31, team = WIDE ? kRowsThreads : 32;
  each_pair<WIDE>(p, [&](int t, int j) {
    const size_t f = (size_t)t * p.k + j;
    const int r = p.row_of[f];
    if ((unsigned)r >= (unsigned)p.n_rows) {
      if (p.dw && me == 0) p.dw[f] = 0.f;
      return;
    }
    const float wj = p.w ? p.w[f] : 1.f;
    const Units q(r, row_bytes);
    const Source<sizeof(T)> d(p.x, p.T, t, q), src(p.dw ? p.rows : p.x, p.n_rows, r, q);
    uint8_t* dst = static_cast<uint8_t*>(p.out) + (size_t)r * row_bytes;
    float dot = 0.f;
    for (int u0 = me; u0 < q.n; u0 += team * 2) {
      uint4 va[2], vb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = u0 + team * i;
        va[i] = vb[i] = make_uint4(0, 0, 0, 0);
        if (u < q.n) {
          va[i] = d.load(q, u);
          if (p.dw) vb[i] = src.load(q, u);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = u0 + team * i;
        if (u >= q.n) break;
        float a[N], b[N];
        widen<T, 16>(va[i], a);
        widen<T, 16>(vb[i], b);
        if (!q.whole(u))
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const int at = q.from(u) + c * (int)sizeof(T);
            if (at < 0 || at >= q.bytes) a[c] = b[c] = 0.f;
          }
#pragma unroll
        for (int c = 0; c < N; ++c) {
          dot = fmaf(a[c], b[c], dot);
          a[c] *= wj;
        }
        if (p.out) store_unit<sizeof(T)>(dst, q, u, narrow<T, 16>(a));
      }
    }
    if (p.dw) {
      dot = pair_sum<WIDE>(dot);
      if (me == 0) p.dw[f] = dot;
    }
  });
}

template <int E>
cudaError_t scatter_odd(RowsDev& p, size_t row_bytes, cudaStream_t s) {
  constexpr int P = 4;
  const long pairs = (long)p.T * p.k;
  p.pad_ctas = pad_ctas(p, kRowsThreads);
  const bool several = (long)row_bytes <= kShortBytes && pairs > 152 * 16;
  const int ctas = (int)std::min<long>((pairs + 7) / 8 / (several ? P : 1) + 1, 1 << 20) + p.pad_ctas;
  if (several) MOE_LAUNCH((k_rows_scatter_odd<E, P>), dim3(ctas), dim3(kRowsThreads), 0, s, p, row_bytes);
  else MOE_LAUNCH((k_rows_scatter_odd<E, 1>), dim3(ctas), dim3(kRowsThreads), 0, s, p, row_bytes);
  return cudaGetLastError();
}
template <typename T>
cudaError_t gather_odd(RowsDev& p, size_t row_bytes, cudaStream_t s) {
  const int units = (int)(row_bytes / 16) + 2, cols = (units + kRowsThreads - 1) / kRowsThreads;
  if (cols > 65535) return cudaErrorInvalidValue;
  const int threads = ((units + cols - 1) / cols + 31) / 32 * 32;  // (no column of CTAs that is nearly empty)
  const dim3 grid(std::min(p.T, std::max(1, 152 * 4096 / (threads * cols))), cols);
  MOE_LAUNCH(k_rows_gather_odd<T>, grid, dim3(threads), 0, s, p, row_bytes);
  return cudaGetLastError();
}
// A launch of a gradient: threads, and CTAs with those that fill the padding.
struct GradShape {
  bool wide;
  int threads, ctas;
};
GradShape grad_shape(RowsDev& p, long row_bytes) {
  GradShape q;
  const long pairs = (long)p.T * p.k;
  q.wide = pairs <= kWidePairs && row_bytes >= kWideBytes;
  q.threads = q.wide ? kRowsThreads : 32 * std::min(p.k, kRowsThreads / 32);
  p.pad_ctas = pad_ctas(p, q.threads);
  q.ctas = (int)std::min<long>(q.wide ? pairs : p.T, 1 << 20) + p.pad_ctas;
  return q;
}
template <typename T>
cudaError_t gather_grad_odd(RowsDev& p, size_t row_bytes, cudaStream_t s) {
  const GradShape q = grad_shape(p, (long)row_bytes);
  if (q.wide) MOE_LAUNCH((k_rows_gather_grad_odd<T, true>), dim3(q.ctas), dim3(q.threads), 0, s, p, row_bytes);
  else MOE_LAUNCH((k_rows_gather_grad_odd<T, false>), dim3(q.ctas), dim3(q.threads), 0, s, p, row_bytes);
  return cudaGetLastError();
}

cudaError_t scatter(RowsDev& p, long row_bytes, cudaStream_t s) {
  p.vpr = (int)(row_bytes / 16);
  // few rows: one vector a lane, so that they spread over more warps
  const long units4 = (long)p.T * ((p.vpr + 127) / 128);
  const bool few = units4 < 152 * 16;
  const int per = few ? 32 : 128;
  p.chunks = (p.vpr + per - 1) / per;
  const long units = (long)p.T * p.chunks;
  p.pad_ctas = pad_ctas(p, kRowsThreads);
  const int ctas = (int)std::min<long>((units + 7) / 8, 1 << 20) + p.pad_ctas;
  if (few) MOE_LAUNCH((k_rows_scatter<1>), dim3(ctas), dim3(kRowsThreads), 0, s, p);
  else MOE_LAUNCH((k_rows_scatter<4>), dim3(ctas), dim3(kRowsThreads), 0, s, p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t gather(RowsDev& p, long row_bytes, cudaStream_t s) {
  p.vpr = (int)(row_bytes / 16);
  const int cols = (p.vpr + kRowsThreads - 1) / kRowsThreads;
  if (cols > 65535) return cudaErrorInvalidValue;
  const dim3 grid(std::min(p.T, std::max(1, 152 * 16 / cols)), cols);
  MOE_LAUNCH((k_rows_gather<T>), grid, dim3(kRowsThreads), 0, s, p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t gather_grad(RowsDev& p, long row_bytes, cudaStream_t s) {
  p.vpr = (int)(row_bytes / 16);
  const GradShape q = grad_shape(p, row_bytes);
  if (q.wide) MOE_LAUNCH((k_rows_gather_grad<T, true>), dim3(q.ctas), dim3(q.threads), 0, s, p);
  else MOE_LAUNCH((k_rows_gather_grad<T, false>), dim3(q.ctas), dim3(q.threads), 0, s, p);
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
  return b % 16 == 0 ? scatter(p, b, s) : elem_bytes == 2 ? scatter_odd<2>(p, b, s) : scatter_odd<4>(p, b, s);
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
  if (b % 16 == 0) return bf16 ? gather<__nv_bfloat16>(p, b, s) : gather<float>(p, b, s);
  return bf16 ? gather_odd<__nv_bfloat16>(p, b, s) : gather_odd<float>(p, b, s);
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
  if (b % 16 == 0) return bf16 ? gather_grad<__nv_bfloat16>(p, b, s) : gather_grad<float>(p, b, s);
  return bf16 ? gather_grad_odd<__nv_bfloat16>(p, b, s) : gather_grad_odd<float>(p, b, s);
}

}  // namespace moe
