// Quantisation to e4m3 by blocks: one fp32 scale per row and 128 consecutive columns.
//
//   a = max |x| over the block;  s = max(a * (1/448), 2^-126), 1 where a = 0
//   q = e4m3(x * (1 / s)), round to nearest even, saturating
// with 1/448 a 32-bit constant and both products and the reciprocal 1 / s (once per block) one
// fp32 rounding each.  A block that holds a NaN gets a NaN scale, one that holds an infinity an
// infinite scale, and all its codes stand for no finite value: a fault upstream stays visible.
// 2^-126 keeps 1 / s finite.
//
// The SiLU form quantises h = SiLU(g) * u of a row [g | u] without storing h.  The scatter form
// serves the expert layer: row t's codes and scales go to the expert-sorted rows of its pairs.
//
// Bound by HBM: an element is read once and leaves as one byte.  8 lanes share a block, 16 elements
// each (two 16-byte loads of bf16, one 16-byte store, the block's maximum in three shuffles), and every
// lane loads kUnroll blocks before it works on the first: with 8 elements a lane and one block at a time
// too few bytes were in flight (8192 x 4096 bf16: 28.9 us, 3.5 TB/s; now 15.4 us, 6.6 TB/s).  The SiLU
// form is bound by the instructions of its exponential and quotient (4099 x 2048: 10.7 us, 3.9 TB/s, 70 %
// of the issue slots).  An approximate quotient takes 8.3 us and moves four times as many codes that lie
// on a border as the arithmetic in 32 bits does by itself: not taken.
#include <algorithm>

#include "moe_align.cuh"
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

// 16 elements, 16-byte loads; widened when they are used
template <typename TIn>
struct Raw16 {
  uint4 v[sizeof(TIn)];
  __device__ __forceinline__ void load(const TIn* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(TIn); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(TIn); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int i) const {
    constexpr int per = 16 / sizeof(TIn);  // elements of one vector
    const uint4& q = v[i / per];
    const int w = (i % per) * sizeof(TIn) / 4;
    const uint32_t u = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
    if constexpr (sizeof(TIn) == 4) return __uint_as_float(u);
    return bf16_bits_to_f32((i & 1) ? (u >> 16) : (u & 0xffffu));
  }
};

// A lane's 16 values of a block that 8 lanes share: the block's scale and the lane's codes.
template <typename Get>
__device__ __forceinline__ uint4 quantise16(Get get, float& s) {
  float v[16], a = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[j] = get(j);
    a = max_nan(a, fabsf(v[j]));
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
  s = block_scale_from_amax(a);
  const float r = 1.0f / s;
  uint4 code;
  code.x = pack_e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
  code.y = pack_e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r);
  code.z = pack_e4m3x4(v[8] * r, v[9] * r, v[10] * r, v[11] * r);
  code.w = pack_e4m3x4(v[12] * r, v[13] * r, v[14] * r, v[15] * r);
  return code;
}

template <typename TIn, bool SILU, bool SCATTER>
__global__ void __launch_bounds__(kQuantThreads) k_quant_block(const QuantDev p) {
  // (dependents launch once this kernel's own wait is over: what came before it is then complete)
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kUnroll = SILU ? 1 : 2;
  const uint32_t l8 = threadIdx.x & 7;
  const uint32_t units = (uint32_t)p.T * (uint32_t)p.nb;
  const uint32_t step = gridDim.x * (kQuantThreads / 8);
  const TIn* x = static_cast<const TIn*>(p.x);
  // (the four blocks of a warp run the same number of rounds: the shuffles name all 32 lanes)
  const uint32_t u0 = blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3);
  for (uint32_t base = u0 & ~3u; base < units; base += kUnroll * step) {
    Raw16<TIn> ra[kUnroll], rb[SILU ? kUnroll : 1];
    uint32_t t[kUnroll], b[kUnroll];
    bool on[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t u = base + (u0 & 3u) + i * step;
      t[i] = u / (uint32_t)p.nb;
      b[i] = u - t[i] * (uint32_t)p.nb;
      const uint32_t c = b[i] * 128u + l8 * 16u;
      on[i] = u < units && c < (uint32_t)p.K;
      if (on[i]) {
        const TIn* row = x + (size_t)t[i] * p.K * (SILU ? 2 : 1) + c;
        ra[i].load(row);
        if constexpr (SILU) rb[i].load(row + p.K);
      } else {
        ra[i].zero();
        if constexpr (SILU) rb[i].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t u = base + (u0 & 3u) + i * step;
      float s;
      const uint4 code = quantise16(
          [&](int j) {
            if constexpr (SILU) return silu(ra[i].get(j)) * rb[i].get(j);
            return ra[i].get(j);
          },
          s);
      const uint32_t c = b[i] * 128u + l8 * 16u;
      if constexpr (SCATTER) {
        if (u < units) {
          for (int j = 0; j < p.k; ++j) {
            const int row = p.inv[(size_t)t[i] * p.k + j];
            if (row < 0) continue;
            if (on[i]) *reinterpret_cast<uint4*>(p.q + (size_t)row * p.K + c) = code;
            if (l8 == 0) p.scale[(size_t)row * p.nb + b[i]] = s;
          }
        }
      } else {
        if (on[i]) *reinterpret_cast<uint4*>(p.q + (size_t)t[i] * p.K + c) = code;
        if (u < units && l8 == 0) p.scale[u] = s;
      }
    }
  }
}

// The scatter form with the permutation in the same launch, for at most 32 pairs: every CTA finds the
// pairs' rows for itself, and one more CTA writes the maps that the products read.  (A launch costs
// such a batch as much as its work does.)
struct AlignQuantDev {
  QuantDev q;
  const int32_t* ids;
  int E, B, skip_minus_one;
  int32_t *sorted, *eids, *meta;
  int* status;
};

__global__ void __launch_bounds__(kQuantThreads) k_align_quant_small(const AlignQuantDev a) {
  // (as k_quant_block: the ids are complete when a dependent starts)
  pdl_wait();
  pdl_launch_dependents();
  const QuantDev& p = a.q;
  const int n = p.T * p.k;
  if (blockIdx.x == gridDim.x - 1) {
    if (threadIdx.x < 32) {
      const SmallGroup g = align_small(a.ids, n, a.E, a.B, a.status, a.skip_minus_one);
      align_small_maps(g, n, a.E, a.B, a.sorted, a.eids, a.meta + META_NPP, nullptr, a.meta, nullptr);
    }
    return;
  }
  __shared__ int s_row[kAlignSmallPairs];
  const int l8 = threadIdx.x & 7;
  const int u = blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3);
  const int t = u / p.nb, b = u - t * p.nb;
  const int c = b * 128 + l8 * 16;
  const bool on = u < p.T * p.nb && c < p.K;
  Raw16<__nv_bfloat16> r16;
  r16.zero();
  if (on) r16.load(static_cast<const __nv_bfloat16*>(p.x) + (size_t)t * p.K + c);
  if (threadIdx.x < 32) {
    const SmallGroup g = align_small(a.ids, n, a.E, a.B, nullptr, 1);
    s_row[threadIdx.x] = g.e >= 0 ? g.slot : -1;
  }
  float s;
  const uint4 code = quantise16([&](int j) { return r16.get(j); }, s);
  __syncthreads();
  if (on) {
    for (int j = 0; j < p.k; ++j) {
      const int row = s_row[t * p.k + j];
      if (row < 0) continue;
      *reinterpret_cast<uint4*>(p.q + (size_t)row * p.K + c) = code;
      if (l8 == 0) p.scale[(size_t)row * p.nb + b] = s;
    }
  }
}

template <typename TIn, bool SILU, bool SCATTER>
cudaError_t launch_inst(const QuantDev& p, cudaStream_t s) {
  const long units = (long)p.T * p.nb;
  if (units >= (1l << 31) - (1l << 24)) return cudaErrorInvalidValue;  // (32-bit unit counts)
  const long blocks = (units + kQuantThreads / 8 - 1) / (kQuantThreads / 8);
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

cudaError_t launch_align_quant_small(const void* x, int T, int K, int k, const int32_t* ids, int E, int B,
                                     int32_t* sorted, int32_t* eids, int32_t* meta, int* status, bool skip_minus_one,
                                     uint8_t* q, float* scale, cudaStream_t s) {
  if ((long)T * k > kAlignSmallPairs) return cudaErrorInvalidValue;
  AlignQuantDev a = {};
  a.q.x = x;
  a.q.q = q;
  a.q.scale = scale;
  a.q.T = T;
  a.q.K = K;
  a.q.nb = (K + 127) / 128;
  a.q.k = k;
  a.ids = ids;
  a.E = E;
  a.B = B;
  a.skip_minus_one = skip_minus_one ? 1 : 0;
  a.sorted = sorted;
  a.eids = eids;
  a.meta = meta;
  a.status = status;
  const int units = T * a.q.nb, per = kQuantThreads / 8;
  MOE_LAUNCH(k_align_quant_small, dim3((units + per - 1) / per + 1), dim3(kQuantThreads), 0, s, a);
  return cudaGetLastError();
}

}  // namespace moe
