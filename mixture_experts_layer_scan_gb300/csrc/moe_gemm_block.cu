// Matrix products of block-scaled e4m3 operands on the tensor cores (tcgen05, sm_103a).
//
//   out[t][n] = sum_b  sa[t][b] * sw[n / 128][b] * sum_{k in block b} a[t][k] * w[n][k]
//
// a [T][K] holds one fp32 scale per row and 128 columns, w [N][K] one per 128 x 128 block.  The
// scales change along K, so they cannot wait for the epilogue: the tensor core sums one block of
// 128 columns (exact products, fp32 sums in tensor memory), and the epilogue warps fold that block
// into fp32 registers with one fma per element, acc += (sa * sw) * block.
//
// Swap-AB orientation: the weight rows fill the tensor core's 128-row M slot and the tokens its N
// slot.  A tile is 256 weight rows (two M = 128 MMAs: D0 and D1) by up to NT tokens; for the first
// expert product the two halves are 128 gate rows and the 128 up rows of the same columns, so a
// tile ends with exactly one 128-column block of the intermediate for each of its tokens: SiLU,
// the block's scale and its codes are formed in the epilogue and no wide intermediate is stored.
//
// Roles (192 threads): warp 0 streams operands by TMA into a ring of shared-memory stages, warp 1
// issues the MMAs into a ring of tensor-memory blocks, warps 2-5 fold the blocks.  Every wait is
// bounded; after one gives up, each role runs on without waiting or storing, so the barriers
// between the epilogue warps stay matched and the kernel ends.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBgThreads = 192;
constexpr int kBgMaxStages = 8;
constexpr int kBgBufs = 4;          // tensor-memory blocks in flight
constexpr int kScaleChunk = 8;      // K blocks whose scale products are staged together
constexpr int kStageTokens = 32;    // tokens of a tile transposed through shared memory at a time

struct BgDev {
  int T, k, E;
  int n_out;            // output columns: N, H, or the intermediate's I
  int kb_total, n_tiles;
  int w_rows, w_pair_off, w_tile_rows;  // weight rows per expert, offset of D1's rows, rows per tile
  int w_scale_rows;     // scale rows per expert
  int s_pair_off;       // offset of D1's scale row from D0's
  int by_block;         // grouped: 1: tiles are the permutation's token blocks, 0: whole experts
  int stages, out_bf16;
  uint32_t stage_bytes, bar_off, scale_off, out_off;
  const float* a_scale;  // [rows][kb_total]
  const float* w_scale;  // [E][w_scale_rows][kb_total]
  const int32_t* sorted;
  const int32_t* eids;
  const int32_t* meta;
  void* out;
  float* out_scale;
  int* status;
};

struct BgTile {
  int e, n, xrow, ntok, npad, wr0;
};

template <int EPI, int NT>
__device__ __forceinline__ int bg_tile_count(const BgDev& p) {
  if constexpr (EPI == BG_EPI_DENSE) return (p.T + NT - 1) / NT * p.n_tiles;
  return (p.by_block ? p.meta[META_NPP] / NT : p.meta[META_NACT]) * p.n_tiles;
}

template <int EPI, int NT>
__device__ __forceinline__ BgTile bg_tile_at(const BgDev& p, int t) {
  BgTile d;
  const int m = t / p.n_tiles;
  d.n = t - m * p.n_tiles;
  if constexpr (EPI == BG_EPI_DENSE) {
    d.e = 0;
    d.xrow = m * NT;
    d.ntok = min(NT, p.T - d.xrow);
  } else if (p.by_block) {
    d.e = p.eids[m];
    d.xrow = m * NT;
    d.ntok = NT;
  } else {
    d.e = p.meta[meta_active(p.E) + m];
    d.xrow = p.meta[meta_offsets(p.E) + d.e];
    d.ntok = p.meta[meta_counts(p.E) + d.e];
  }
  d.npad = (d.ntok + 15) & ~15;
  d.wr0 = d.e * p.w_rows + d.n * p.w_tile_rows;
  return d;
}

// (a0, a1) = (s0, s1) * (d0, d1) + (a0, a1): one packed instruction, each half one fp32 rounding
__device__ __forceinline__ void fma2(float2& a, float s0, float s1, float d0, float d1) {
  uint64_t av, sv, dv;
  asm("mov.b64 %0, {%1, %2};" : "=l"(av) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(sv) : "f"(s0), "f"(s1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(dv) : "f"(d0), "f"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(av) : "l"(sv), "l"(dv));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(av));
}

// One token's 256 sums (shared memory, staged as [token][256]) by one warp.
template <int EPI>
__device__ __forceinline__ void bg_store_row(const BgDev& p, const BgTile& d, const float* row, int c, int lane) {
  const float4 v0 = *reinterpret_cast<const float4*>(row + 4 * lane);
  const float4 v1 = *reinterpret_cast<const float4*>(row + 128 + 4 * lane);
  if constexpr (EPI == BG_EPI_G1) {
    const float h0 = silu(v0.x) * v1.x, h1 = silu(v0.y) * v1.y, h2 = silu(v0.z) * v1.z, h3 = silu(v0.w) * v1.w;
    float a = max_nan(max_nan(fabsf(h0), fabsf(h1)), max_nan(fabsf(h2), fabsf(h3)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
    const float s = block_scale_from_amax(a);
    const float r = 1.0f / s;
    const size_t xr = (size_t)(d.xrow + c);
    reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + xr * p.n_out + (size_t)d.n * 128)[lane] =
        pack_e4m3x4(h0 * r, h1 * r, h2 * r, h3 * r);
    if (lane == 0) p.out_scale[xr * (p.n_out / 128) + d.n] = s;
  } else if constexpr (EPI == BG_EPI_G2) {
    const int f = p.sorted[d.xrow + c];
    if (f >= p.T * p.k) return;
    float* y = static_cast<float*>(p.out) + (size_t)f * p.n_out + (size_t)d.n * 256 + 4 * lane;
    *reinterpret_cast<float4*>(y) = v0;
    if (d.n * 256 + 128 < p.n_out) *reinterpret_cast<float4*>(y + 128) = v1;
  } else {
    const size_t o = (size_t)(d.xrow + c) * p.n_out;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const float4 v = hf ? v1 : v0;
      const int n = d.n * 256 + hf * 128 + 4 * lane;
      if (p.n_out % 4 == 0) {
        if (n >= p.n_out) continue;
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o + n) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o + n) = v;
      } else {
        const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (n + i >= p.n_out) continue;
          if (p.out_bf16)
            static_cast<__nv_bfloat16*>(p.out)[o + n + i] = __float2bfloat16_rn(e[i]);
          else
            static_cast<float*>(p.out)[o + n + i] = e[i];
        }
      }
    }
  }
}

template <int EPI, int NT>
__global__ void __launch_bounds__(kBgThreads, 1)
    k_gemm_block(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const BgDev p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + p.bar_off;
  const uint32_t bar_empty = bar_full + 8 * kBgMaxStages;
  const uint32_t bar_tfull = bar_empty + 8 * kBgMaxStages;
  const uint32_t bar_tempty = bar_tfull + 8 * kBgBufs;
  const uint32_t bar_drain = bar_tempty + 8 * kBgBufs;
  const uint32_t bar_exit = bar_drain + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.bar_off + 8 * (2 * kBgMaxStages + 2 * kBgBufs + 2));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t kCols = 2 * NT * kBgBufs;  // 128, 256 or 512: a power of two
  constexpr uint32_t kHalfBytes = 128 * 128;    // 128 weight rows of one K block

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < kBgBufs; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, 4);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_exit, kBgThreads / 32);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kCols);
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  const int ntiles = bg_tile_count<EPI, NT>(p);

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
      const BgTile d = bg_tile_at<EPI, NT>(p, t);
      for (int kb = 0; kb < p.kb_total; ++kb) {
        if (!mbar_wait_all(bar_empty + 8 * stage, phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t sw = sbase + stage * p.stage_bytes, fb = bar_full + 8 * stage;
          mbar_arrive_expect_tx(fb, 2 * kHalfBytes + (uint32_t)d.npad * 128u);
          tma_load_2d(sw, &tmW, kb * 128, d.wr0, fb);
          tma_load_2d(sw + kHalfBytes, &tmW, kb * 128, d.wr0 + p.w_pair_off, fb);
          for (int r = 0; r < d.npad; r += 16)
            tma_load_2d(sw + 2 * kHalfBytes + (uint32_t)r * 128u, &tmX, kb * 128, d.xrow + r, fb);
        }
        __syncwarp();
        ++issued;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      pdl_launch_dependents();
      if (!ok) {  // let the copies already in flight land before the CTA exits
        const uint32_t first = issued > (uint32_t)p.stages ? issued - p.stages : 0u;
        for (uint32_t i = first; i < issued; ++i)
          mbar_wait_drain(bar_full + 8 * (i % p.stages), (i / p.stages) & 1u, 100000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    int stage = 0, buf = 0;
    uint32_t phase = 0, buf_phase = 0;
    bool ok = true, any = false;
    for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
      const BgTile d = bg_tile_at<EPI, NT>(p, t);
      const uint32_t idesc = idesc_make(128, d.npad, true);
      for (int kb = 0; kb < p.kb_total; ++kb) {
        if (!mbar_wait_all(bar_tempty + 8 * buf, buf_phase ^ 1u, abort_flag, p.status) ||
            !mbar_wait_all(bar_full + 8 * stage, phase, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sw = sbase + stage * p.stage_bytes;
          const uint32_t dt = tmem_base + (uint32_t)(buf * 2 * NT);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bdesc = sdesc_k_sw128(sw + 2 * kHalfBytes + kk * 32);
            tc_mma<true>(dt, sdesc_k_sw128(sw + kk * 32), bdesc, idesc, kk > 0);
            tc_mma<true>(dt + NT, sdesc_k_sw128(sw + kHalfBytes + kk * 32), bdesc, idesc, kk > 0);
          }
          tc_commit(bar_empty + 8 * stage);
          tc_commit(bar_tfull + 8 * buf);
        }
        __syncwarp();
        any = true;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == kBgBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
    }
    if (!ok && any) {  // the tensor core must be idle before tensor memory is freed
      if (lane == 0) tc_commit(bar_drain);
      __syncwarp();
      mbar_wait_drain(bar_drain, 0, 100000000ull);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue (warps 2..5): fold the blocks, then the outputs ----------------
    const int q = warp & 3;          // tensor-memory lane quadrant this warp may read
    const int lrow = q * 32 + lane;  // weight row of this thread in D0 and in D1
    const int tid = threadIdx.x - 64;
    float* sc = reinterpret_cast<float*>(smem + p.scale_off);  // [2][2][kScaleChunk][NT]
    float* st = reinterpret_cast<float*>(smem + p.out_off);    // [kStageTokens][256]
    constexpr int kSet = kScaleChunk * NT;                     // scale products of one chunk and half
    constexpr int kPer = kSet / 128;
    const int lane_kb = tid % kScaleChunk, lane_c = tid / kScaleChunk;  // this thread's first scale of a chunk
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
      const BgTile d = bg_tile_at<EPI, NT>(p, t);
      const int srow = d.n * (p.w_tile_rows / 128);
      const float* ws0 = p.w_scale + ((size_t)d.e * p.w_scale_rows + srow) * p.kb_total;
      const float* ws1 =
          p.w_scale + ((size_t)d.e * p.w_scale_rows + min(srow + p.s_pair_off, p.w_scale_rows - 1)) * p.kb_total;
      // scales of the next chunk, one K block and every 16th token to a thread
      float ra[kPer], r0 = 0.0f, r1 = 0.0f;
      auto fetch = [&](int kb) {
        const bool in = kb + lane_kb < p.kb_total;
        r0 = in ? ws0[kb + lane_kb] : 0.0f;
        r1 = in ? ws1[kb + lane_kb] : 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = lane_c + i * (128 / kScaleChunk);
          ra[i] = (in && c < d.ntok) ? p.a_scale[(size_t)(d.xrow + c) * p.kb_total + kb + lane_kb] : 0.0f;
        }
      };
      float2 acc0[NT / 2], acc1[NT / 2];
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) acc0[i] = acc1[i] = make_float2(0.0f, 0.0f);
      fetch(0);
      for (int kc = 0, par = 0; kc < p.kb_total; kc += kScaleChunk, par ^= 1) {
        float* s0 = sc + par * 2 * kSet;
        float* s1 = s0 + kSet;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = lane_c + i * (128 / kScaleChunk);
          s0[lane_kb * NT + c] = ra[i] * r0;
          s1[lane_kb * NT + c] = ra[i] * r1;
        }
        named_bar_sync(1, 128);
        if (kc + kScaleChunk < p.kb_total) fetch(kc + kScaleChunk);
        const int kn = min(kScaleChunk, p.kb_total - kc);
        for (int kb = 0; kb < kn; ++kb) {
          ok = ok && mbar_wait_all(bar_tfull + 8 * buf, buf_phase, abort_flag, p.status);
          if (ok) {
            tc_fence_after();
            const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * 2 * NT);
#pragma unroll
            for (int c0 = 0; c0 < NT; c0 += 16) {
              if (c0 < d.npad) {
                float v0[16], v1[16];
                tmem_ld16(tb + c0, v0);
                tmem_ld16(tb + NT + c0, v1);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  const float4 f0 = *reinterpret_cast<const float4*>(s0 + kb * NT + c0 + j);
                  const float4 f1 = *reinterpret_cast<const float4*>(s1 + kb * NT + c0 + j);
                  fma2(acc0[(c0 + j) / 2], f0.x, f0.y, v0[j], v0[j + 1]);
                  fma2(acc0[(c0 + j) / 2 + 1], f0.z, f0.w, v0[j + 2], v0[j + 3]);
                  fma2(acc1[(c0 + j) / 2], f1.x, f1.y, v1[j], v1[j + 1]);
                  fma2(acc1[(c0 + j) / 2 + 1], f1.z, f1.w, v1[j + 2], v1[j + 3]);
                }
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_tempty + 8 * buf);
          }
          if (++buf == kBgBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      // transpose kStageTokens tokens at a time: thread = weight row -> warp = token
#pragma unroll
      for (int c0 = 0; c0 < NT; c0 += kStageTokens) {
        if (c0 < d.ntok) {
#pragma unroll
          for (int c = 0; c < (NT < kStageTokens ? NT : kStageTokens); c += 2) {
            const int i = (c0 + c) / 2;
            st[c * 256 + lrow] = acc0[i].x;
            st[(c + 1) * 256 + lrow] = acc0[i].y;
            st[c * 256 + 128 + lrow] = acc1[i].x;
            st[(c + 1) * 256 + 128 + lrow] = acc1[i].y;
          }
          named_bar_sync(1, 128);
          if (ok)
            for (int c = c0 + q; c < min(d.ntok, c0 + kStageTokens); c += 4)
              bg_store_row<EPI>(p, d, st + (c - c0) * 256, c, lane);
          named_bar_sync(1, 128);
        }
      }
    }
  }

  // Each warp reports the end of its role on an mbarrier; warp 1 frees tensor memory once every
  // warp has.
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar_exit);
  if (warp == 1) {
    mbar_wait_drain(bar_exit, 0, 2 * kWaitLimitNs);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
}

template <int EPI, int NT>
cudaError_t launch_bg(const CUtensorMap& mw, const CUtensorMap& mx, BgDev p, long tiles, int sms, cudaStream_t s) {
  p.stage_bytes = 2u * 128u * 128u + (uint32_t)NT * 128u;
  const uint32_t bar_bytes = 8 * (2 * kBgMaxStages + 2 * kBgBufs + 2) + 16;
  const uint32_t scale_bytes = 2u * 2u * kScaleChunk * NT * 4u;
  const uint32_t out_bytes = (uint32_t)std::min(NT, kStageTokens) * 256u * 4u;
  p.stages = std::min<int>(kBgMaxStages, (227 * 1024 - 1024 - bar_bytes - scale_bytes - out_bytes) / p.stage_bytes);
  p.out_off = (uint32_t)p.stages * p.stage_bytes;
  p.scale_off = p.out_off + out_bytes;
  p.bar_off = p.scale_off + scale_bytes;
  const size_t smem = 1024 + (size_t)p.bar_off + bar_bytes;
  auto kern = k_gemm_block<EPI, NT>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int grid = (int)std::max<long>(1, std::min<long>(tiles, sms));
  return launch_pdl(kern, dim3(grid), dim3(kBgThreads), smem, s, mw, mx, p);
}

template <int EPI>
cudaError_t launch_bg_nt(const CUtensorMap& mw, const CUtensorMap& mx, const BgDev& p, int nt, long tiles, int sms,
                         cudaStream_t s) {
  if (nt == 16) return launch_bg<EPI, 16>(mw, mx, p, tiles, sms, s);
  if (nt == 32) return launch_bg<EPI, 32>(mw, mx, p, tiles, sms, s);
  if (nt == 64) return launch_bg<EPI, 64>(mw, mx, p, tiles, sms, s);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gemm_block(const BlockGemmArgs& a, cudaStream_t s) {
  CUtensorMap mw, mx;
  const uint64_t x_rows = a.epi == BG_EPI_DENSE ? (uint64_t)a.T : (uint64_t)a.cap;
  if (!make_tensor_map_2d(&mw, a.w, 1, (uint64_t)a.K, (uint64_t)a.E * a.w_rows, 128u) ||
      !make_tensor_map_2d(&mx, a.x, 1, (uint64_t)a.K, x_rows, 16u))
    return cudaErrorInvalidValue;
  BgDev p = {};
  p.T = a.T;
  p.k = a.k;
  p.E = a.E;
  p.n_out = a.n_out;
  p.kb_total = (a.K + 127) / 128;
  p.w_rows = a.w_rows;
  p.w_scale_rows = (a.w_rows + 127) / 128;
  if (a.epi == BG_EPI_G1) {
    p.n_tiles = a.n_out / 128;
    p.w_pair_off = a.n_out;
    p.w_tile_rows = 128;
    p.s_pair_off = a.n_out / 128;
  } else {
    p.n_tiles = (a.n_out + 255) / 256;
    p.w_pair_off = 128;
    p.w_tile_rows = 256;
    p.s_pair_off = 1;
  }
  p.by_block = a.by_block ? 1 : 0;
  p.out_bf16 = a.out_bf16 ? 1 : 0;
  p.a_scale = a.a_scale;
  p.w_scale = a.w_scale;
  p.sorted = a.sorted;
  p.eids = a.eids;
  p.meta = a.meta;
  p.out = a.out;
  p.out_scale = a.out_scale;
  p.status = a.status;
  if (a.epi == BG_EPI_DENSE) {
    const long tiles = ((long)a.T + a.nt - 1) / a.nt * p.n_tiles;
    return launch_bg_nt<BG_EPI_DENSE>(mw, mx, p, a.nt, tiles, a.num_sms, s);
  }
  const long groups = a.by_block ? (long)a.cap / a.nt : std::min<long>(a.E, (long)a.T * a.k);
  if (a.epi == BG_EPI_G1) return launch_bg_nt<BG_EPI_G1>(mw, mx, p, a.nt, groups * p.n_tiles, a.num_sms, s);
  return launch_bg_nt<BG_EPI_G2>(mw, mx, p, a.nt, groups * p.n_tiles, a.num_sms, s);
}

}  // namespace moe
