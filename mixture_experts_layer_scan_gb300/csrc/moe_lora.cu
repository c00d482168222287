// Low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + s[l] B_l (A_l x_t),  l = ids[t];  out[t] = base[t] where ids[t] = -1
//
// Little work (lora_plan says how much): two launches on the CUDA cores, h = s A x (fp32, in the workspace), then out = base + B h, a
// token at a time (its adapter's rows come from L2 where tokens share them).
//
// More work: the tokens are sorted by adapter (the permutation of the expert layer, an adapter in the place of an
// expert, blocks of 128 tokens, those without one behind), and both products run on the tensor cores, kind::f16 with fp32 sums:
//   shrink   a CTA to a block and a run of K: D[128 tokens x r] += X A^T over blocks of 64 K, A by TMA, X's rows by
//            16-byte asynchronous copies (TMA gathers of four rows of 128 bytes took about 1 us for a block);
//            the CTAs of a block are a cluster and add up their fp32 sums in the order of K through distributed
//            shared memory: h = s A x, as bf16 parts that add up to it (2 for a bf16 output: off by 2^-16 of
//            h at most; 3 for an fp32 one: all of its bits)
//   expand   persistent over (block, tile of 256 bytes of output columns): h becomes the A operand in tensor
//            memory, B's rows come by TMA, and the epilogue adds the base
// A token's row of D depends on that token alone, so what padding rows of a block hold does not matter.
// Bound by HBM: 8192 tokens of rank 64 through 4096 x 8192 take 85 us, 50 of them the expand kernel's tiles at 5.4 TB/s;
// 777 of rank 32 through 2040 x 5000 28, mostly what three dependent launches cost.
// Two launches rather than clusters that exchange h: a CTA that holds tensor memory never waits for another
// CTA, so calls on several streams cannot block one another.
#include <algorithm>
#include <type_traits>

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

// Products of eight bf16 pairs in fp32, added to acc in their order.
__device__ __forceinline__ float dot8(const uint4& a, const float (&fb)[8], float acc) {
  float fa[8];
  widen<__nv_bfloat16, 16>(a, fa);
#pragma unroll
  for (int c = 0; c < 8; ++c) acc = fmaf(fa[c], fb[c], acc);
  return acc;
}

// A CTA to a token and eight rows of its A: a warp takes every eighth run of 256 columns for all of the rows
// (eight row loads of a lane in flight beside one of x), and the warps' sums meet in shared memory.
constexpr int kShrinkRows = 8;
__global__ void __launch_bounds__(256) k_lora_shrink(const LoraDev p) {
  pdl_enter();
  __shared__ float s[8][kShrinkRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = blockIdx.y * kShrinkRows;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int l = p.ids[t];
    if (l >= p.L || l < 0) {
      if (l != -1 && threadIdx.x == 0 && blockIdx.y == 0) report(p.status, MOE_ERR_DEVICE_INDEX);
      continue;
    }
    const int vecs = p.K / 8;
    const uint4* xv = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.K);
    const uint4* av = reinterpret_cast<const uint4*>(p.a + ((size_t)l * p.r + i0) * p.K);
    float acc[kShrinkRows] = {};
#pragma unroll 2
    for (int v = warp * 32 + lane; v < vecs; v += 256) {
      uint4 a[kShrinkRows];
      const uint4 x = xv[v];
#pragma unroll
      for (int i = 0; i < kShrinkRows; ++i) a[i] = av[(size_t)i * vecs + v];
      float fx[8];
      widen<__nv_bfloat16, 16>(x, fx);
#pragma unroll
      for (int i = 0; i < kShrinkRows; ++i) acc[i] = dot8(a[i], fx, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < kShrinkRows; ++i)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    __syncthreads();  // (the token before has been read)
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < kShrinkRows; ++i) s[warp][i] = acc[i];
    __syncthreads();
    if (threadIdx.x < kShrinkRows) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) sum += s[w][threadIdx.x];
      p.h[(size_t)t * p.r + i0 + threadIdx.x] = p.scale ? sum * p.scale[l] : sum;
    }
  }
}

// A CTA to a token and a run of output columns: G lanes share a column's row of B (16 bytes each),
// and a warp walks 32 / G columns at a time, kExpandUnroll steps in flight.
constexpr int kExpandUnroll = 8;
constexpr int kExpandStep = 1 << 23;  // columns from a CTA's step to its next, at most (N is below 2^31 - 2^24)
template <typename T, int G>
__global__ void __launch_bounds__(256) k_lora_expand(const LoraDev p) {
  pdl_enter();
  constexpr int kCols = 32 / G;                      // columns of a warp's step
  constexpr int kRun = 8 * kCols * kExpandUnroll;    // columns of a CTA's step
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane % G;
  const int chunks = p.r / 8;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int l = p.ids[t];
    const bool on = l >= 0 && l < p.L && g < chunks;
    float h[8] = {};
    if (on) {
      const float4* hp = reinterpret_cast<const float4*>(p.h + (size_t)t * p.r + g * 8);
      const float4 a = hp[0], b = hp[1];
      h[0] = a.x; h[1] = a.y; h[2] = a.z; h[3] = a.w;
      h[4] = b.x; h[5] = b.y; h[6] = b.z; h[7] = b.w;
    }
    const uint4* bv = reinterpret_cast<const uint4*>(p.b + (size_t)max(l, 0) * p.N * p.r);
    for (int n0 = blockIdx.y * kRun + warp * kCols * kExpandUnroll + lane / G; n0 - lane / G < p.N; n0 += gridDim.y * kRun) {
      uint4 w[kExpandUnroll];
      float base[kExpandUnroll];
#pragma unroll
      for (int u = 0; u < kExpandUnroll; ++u) {
        const int n = n0 + u * kCols;
        w[u] = make_uint4(0, 0, 0, 0);
        base[u] = 0.f;
        if (n < p.N) {
          if (on) w[u] = bv[(size_t)n * chunks + g];
          if (p.base && g == 0) base[u] = to_f32(static_cast<const T*>(p.base)[(size_t)t * p.N + n]);
        }
      }
#pragma unroll
      for (int u = 0; u < kExpandUnroll; ++u) {
        float d = dot8(w[u], h, 0.f);
#pragma unroll
        for (int o = 1; o < G; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        const int n = n0 + u * kCols;
        if (g == 0 && n < p.N) {
          const size_t at = (size_t)t * p.N + n;
          if constexpr (sizeof(T) == 4) static_cast<float*>(p.out)[at] = base[u] + d;
          else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(base[u] + d);
        }
      }
    }
  }
}

template <typename T, int G>
cudaError_t launch_few(const LoraDev& p, cudaStream_t s) {
  constexpr int kRun = 8 * (32 / G) * kExpandUnroll;
  const int rows = std::min(p.T, 1 << 16);
  MOE_LAUNCH(k_lora_shrink, dim3(rows, p.r / kShrinkRows), dim3(256), 0, s, p);
  const int runs = std::min((p.N + kRun - 1) / kRun, std::min(kExpandStep / kRun, 65535));
  MOE_LAUNCH((k_lora_expand<T, G>), dim3(rows, runs), dim3(256), 0, s, p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_few(const LoraDev& p, cudaStream_t s) {
  const int chunks = p.r / 8;
  return chunks <= 1   ? launch_few<T, 1>(p, s)
         : chunks <= 2 ? launch_few<T, 2>(p, s)
         : chunks <= 4 ? launch_few<T, 4>(p, s)
         : chunks <= 8 ? launch_few<T, 8>(p, s)
                       : launch_few<T, 16>(p, s);
}

// ---------------------------------------------------------------------------
// tensor cores
// ---------------------------------------------------------------------------
constexpr int kBlk = 128;          // tokens of a block
constexpr int kMaxStages = 6;
constexpr int kBufs = 2;           // output tiles in tensor memory
constexpr int kSegBytes = 128;     // of a row of the output tile, half of which a warp takes
constexpr int kShrinkThreads = 192;  // A's producer, MMA, 4 warps that load x and store the sums
constexpr int kExpandThreads = 576;  // producer, MMA, two sets of 8 epilogue warps
constexpr int kExpandCols = 512;
constexpr int kSlots = 152 * 2;    // CTAs of the shrink kernel that are resident together
constexpr int kMaxSplits = 8;
constexpr int kMaxParts = 3;
constexpr int kBaseStages = 4;     // tiles of base in shared memory (two of each set of epilogue warps)
constexpr int kPieceRow = kSegBytes + 16;  // bytes from row to row of a warp's piece: no bank is met twice
constexpr int kPieceBytes = 32 * kPieceRow;

struct LoraTcDev {
  int T, K, N, r, L;
  int rn;                 // rank rounded up to 16
  int nblk_max;
  int kb_total, kb_per, splits;
  int stages;
  uint32_t stage_bytes, bar_off, base_off;
  int n_tiles;
  const __nv_bfloat16* x;
  const int32_t *sorted, *eids, *meta;
  const float* scale;
  int parts;              // bf16 parts of h
  uint4* hp;              // h as the expand kernel takes it: [block][part * rn / 8][128 rows], 8 columns each
  const void* base;
  void* out;
  int* status;
};

// Blocks of tokens with an adapter; those without one are the last group of the permutation.
__device__ __forceinline__ int lora_blocks(const LoraTcDev& p) { return p.meta[meta_offsets(p.L + 1) + p.L] / kBlk; }

struct TcBars {
  uint32_t full, empty, tfull, tempty, done, drain, exit;
  uint32_t* slot;
  volatile int* abort;
};
__device__ __forceinline__ TcBars tc_bars(uint8_t* smem, uint32_t off) {
  TcBars b;
  b.full = smem_u32(smem) + off;
  b.empty = b.full + 8 * kMaxStages;
  b.tfull = b.empty + 8 * kMaxStages;
  b.tempty = b.tfull + 8 * kBufs;
  b.done = b.tempty + 8 * kBufs;
  b.drain = b.done + 8;
  b.exit = b.drain + 8;
  b.slot = reinterpret_cast<uint32_t*>(smem + off + 8 * (2 * kMaxStages + 2 * kBufs + 3));
  b.abort = reinterpret_cast<volatile int*>(b.slot + 1);
  return b;
}
constexpr uint32_t kBarBytes = 8 * (2 * kMaxStages + 2 * kBufs + 3) + 16;

// Barriers and tensor memory of a CTA; every thread.  Arrivals of `full` and `done` as given.
__device__ __forceinline__ uint32_t tc_setup(const TcBars& b, int cols, int full_count, int done_count) {
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(b.full + 8 * s, full_count);
      mbar_init(b.empty + 8 * s, 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(b.tfull + 8 * i, 1);
      mbar_init(b.tempty + 8 * i, 8);
    }
    mbar_init(b.done, done_count);
    mbar_init(b.drain, 1);
    mbar_init(b.exit, blockDim.x / 32);
    *b.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(b.slot), cols);
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  return *b.slot;
}

// The end of every warp's role; warp 1 frees tensor memory once every warp is there.
__device__ __forceinline__ void tc_finish(const TcBars& b, uint32_t tmem, int cols) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(b.exit);
  if ((threadIdx.x >> 5) == 1) {
    mbar_wait_drain(b.exit, 0, 2 * kWaitLimitNs);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

__device__ __forceinline__ int pow2_cols(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : 128; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {  // (zeros where !in)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// What is left of h behind its part.
__device__ __forceinline__ float lora_rest(float h, float part) {
  if (isinf(part)) return copysignf(1.0f, part);
  const float rest = h - part;
  return rest == 0.0f ? part * 0x1p-32f : rest;
}

// 8 columns of a row of h from c on, scaled and as `parts` bf16 numbers that add up to each: all but the last cut off, not
// rounded, so that none of a finite h is infinite and all have its sign.  Where nothing is left for one, it is 2^-32 of the
// one before (of an infinite one 1), so that with an infinite b no product is NaN (an h below 2^-62 still gives one).
__device__ __forceinline__ void lora_store_h(const LoraTcDev& p, int blk, int row, int c, float s, float (&h)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = c + e < p.r ? h[e] * s : 0.f;
  uint4* dst = p.hp + ((size_t)blk * p.parts * (p.rn / 8) + c / 8) * kBlk + row;
  for (int part = 0; part < p.parts; ++part) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = part + 1 < p.parts ? __byte_perm(__float_as_uint(h[2 * e]), __float_as_uint(h[2 * e + 1]), 0x7632)
                                : pack_bf16x2(h[2 * e], h[2 * e + 1]);
      const float lo = bf16_bits_to_f32(u[e] & 0xffffu), hi = bf16_bits_to_f32(u[e] >> 16);
      h[2 * e] = lora_rest(h[2 * e], lo);
      h[2 * e + 1] = lora_rest(h[2 * e + 1], hi);
    }
    dst[(size_t)part * (p.rn / 8) * kBlk] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

template <int STAGES>
__global__ void __launch_bounds__(kShrinkThreads)
    k_lora_shrink_tc(const __grid_constant__ CUtensorMap tmA, const LoraTcDev p) {
  pdl_wait();
  const int nblk = lora_blocks(p);
  const int blk = blockIdx.x / p.splits, split = blockIdx.x - blk * p.splits;
  if (blk >= nblk) return;  // (a whole cluster)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const TcBars b = tc_bars(smem, p.bar_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = pow2_cols(p.rn);
  const uint32_t tmem = tc_setup(b, cols, 5, 1);
  // Dependents launch once every CTA here holds its tensor memory: the expand kernel's CTAs take theirs before they wait
  // for this kernel.
  pdl_launch_dependents();
  const int kb0 = split * p.kb_per, kb1 = min(kb0 + p.kb_per, p.kb_total);
  constexpr uint32_t kXBytes = kBlk * 128;

  if (warp == 0) {
    const int l = p.eids[blk];
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_all(b.empty + 8 * stage, phase ^ 1u, b.abort, p.status)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        const uint32_t fb = b.full + 8 * stage;
        mbar_arrive_expect_tx(fb, (uint32_t)p.r * 128u);
        tma_load_2d(sbase + stage * p.stage_bytes + kXBytes, &tmA, kb * 64, l * p.r, fb);
      }
      __syncwarp();
      ++issued;
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {  // let the copies already in flight land before the CTA exits
      const uint32_t from = issued > (uint32_t)STAGES ? issued - STAGES : 0u;
      for (uint32_t i = from; i < issued; ++i)
        mbar_wait_drain(b.full + 8 * (i % STAGES), (i / STAGES) & 1u, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_make(kBlk, p.rn, false);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait_one(b.full + 8 * stage, phase, b.abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sx = sbase + stage * p.stage_bytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma<false>(tmem, sdesc_k_sw128(sx + kk * 32), sdesc_k_sw128(sx + kXBytes + kk * 32), idesc,
                        kb > kb0 || kk > 0);
        tc_commit(b.empty + 8 * stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) {
        tc_commit(b.done);
      } else {  // the tensor core must be idle before tensor memory is freed
        tc_commit(b.drain);
        mbar_wait_drain(b.drain, 0, 100000000ull);
      }
    }
    __syncwarp();
  } else {
    // x: 8 lanes to the 128 bytes of a row, 16 rows from one of a thread's pieces to the next
    const int tid = threadIdx.x - 64, r0 = tid >> 3, chunk = tid & 7;
    const __nv_bfloat16* row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = p.sorted[(size_t)blk * kBlk + r0 + 16 * i];
      row[i] = (unsigned)t < (unsigned)p.T ? p.x + (size_t)t * p.K + chunk * 8 : nullptr;
    }
    const uint32_t at = sbase + (uint32_t)r0 * 128u + (uint32_t)((chunk ^ (r0 & 7)) * 16);  // 128-byte swizzle
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // (a stage is handed over while kLag younger ones load; one more may then be with the tensor core)
    constexpr int kLag = STAGES - 2;
    const int n = kb1 - kb0;
    for (int i = 0; i < n + kLag; ++i) {
      if (i < n) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_one(b.empty + 8 * stage, phase ^ 1u, b.abort, p.status));
        if (ok) {
          const int k = (kb0 + i) * 64;
          const bool in = k + chunk * 8 < p.K;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (row[c]) cp_async16(at + stage * p.stage_bytes + c * 16 * 128, in ? row[c] + k : row[c], in);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      cp_async_commit();
      if (i >= kLag) {  // the oldest stage's copies are there: hand it to the tensor core
        cp_async_wait<kLag>();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.full + 8 * ((i - kLag) % STAGES));
      }
    }
    const int q = warp & 3;
    ok = __all_sync(0xffffffffu, mbar_wait_one(b.done, 0, b.abort, p.status)) && ok;
    tc_fence_after();
    const int me = q * 32 + lane;
    // (the ring is idle: its memory takes the sums, [rn / 4][128 rows] float4)
    if (ok) {
      for (int c = 0; c < p.rn; c += 16) {
        float v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sts_v4(sbase + ((uint32_t)(c / 4 + i) * kBlk + me) * 16,
                 make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                            __float_as_uint(v[4 * i + 3])));
      }
    }
  }
  // Tensor memory is given back before this CTA waits for others of its cluster: none that needs some ever waits
  // for one that waits.
  tc_finish(b, tmem, cols);
  __syncwarp();
  cluster_sync_all();
  if (warp >= 2) {
    const int me = (warp & 3) * 32 + lane;
    const float scale = p.scale ? p.scale[p.eids[blk]] : 1.0f;
    for (int c = split * 8; c < p.rn; c += p.splits * 8) {
      const uint32_t at = sbase + ((uint32_t)(c / 4) * kBlk + me) * 16;
      float4 u[kMaxSplits], v[kMaxSplits];
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < p.splits) {
          const uint32_t from = mapa_shared(at, r);
          u[r] = ld_cluster_f32x4(from);
          v[r] = ld_cluster_f32x4(from + kBlk * 16);
        }
      float h[8] = {};
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < p.splits) {
          h[0] += u[r].x; h[1] += u[r].y; h[2] += u[r].z; h[3] += u[r].w;
          h[4] += v[r].x; h[5] += v[r].y; h[6] += v[r].z; h[7] += v[r].w;
        }
      lora_store_h(p, blk, me, c, scale, h);
    }
  }
  __syncwarp();
  cluster_sync_all();  // (no CTA leaves while another reads its sums)
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// The tiles of one CTA: an equal run of the (block, tile) pairs.  (Neighbouring tiles to neighbouring CTAs, so that
// what is in flight lies together in memory, was slower: a call of 8192 tokens of rank 64 took 120 us where it then took 92.)
struct LoraWalk {
  int blk, tile, at, end, tiles;
  __device__ __forceinline__ LoraWalk(const LoraTcDev& p, int nblk) {  // (of the first nblk blocks)
    tiles = p.n_tiles;
    const long total = (long)nblk * tiles;
    at = (int)(total * blockIdx.x / gridDim.x);
    end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    blk = at / tiles;
    tile = at - blk * tiles;
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ void next() {
    ++at;
    if (++tile == tiles) {
      tile = 0;
      ++blk;
    }
  }
};

// Persistent; a CTA's two sets of epilogue warps take its tiles in turn (a warp's way through a tile is a chain
// of latencies: a call of 8192 tokens of rank 64 took 113 us with one set, 92 with two).  A
// warp owns 32 rows x 128 bytes of a tile: it copies that piece of base into shared memory ahead of time,
// adds D there with a row to a thread, and stores it with 8 lanes to a row, without a barrier beyond its own.
template <typename T, int PARTS>
__global__ void __launch_bounds__(kExpandThreads)
    k_lora_expand_tc(const __grid_constant__ CUtensorMap tmB, const LoraTcDev p) {
  constexpr int kHalf = kSegBytes / sizeof(T);  // columns of a warp's piece
  constexpr int kNT = 2 * kHalf;                // columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const TcBars b = tc_bars(smem, p.bar_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = tc_setup(b, kExpandCols, 1, 16);
  // (every thread, before it reads anything: the permutation and base are of kernels before the preceding one, and only
  // this wait makes them visible here; reading them ahead of it took 777 tokens from 27.9 to 26.8 us, 8192 from 84.5 to 83.3)
  pdl_wait();
  const int nblk = lora_blocks(p);
  const uint32_t hcols = (uint32_t)(p.rn / 2);  // columns of one part of h
  const uint32_t h0 = tmem + kBufs * kNT;
  const int kboxes = (p.r + 63) / 64;
  constexpr uint32_t kBoxBytes = kNT * 128;
  LoraWalk w(p, p.base == p.out ? nblk : p.meta[META_NBLK]);  // (in place, rows without an adapter are done)

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (; w.more() && w.blk < nblk; w.next()) {
      if (!mbar_wait_all(b.empty + 8 * stage, phase ^ 1u, b.abort, p.status)) {
        ok = false;
        break;
      }
      const int row = p.eids[w.blk] * p.N + w.tile * kNT;
      if (elect_one()) {
        const uint32_t sw = sbase + stage * p.stage_bytes, fb = b.full + 8 * stage;
        mbar_arrive_expect_tx(fb, (uint32_t)kboxes * kBoxBytes);
        for (int x = 0; x < kboxes; ++x) tma_load_2d(sw + x * kBoxBytes, &tmB, x * 64, row, fb);
      }
      __syncwarp();
      ++issued;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    pdl_launch_dependents();
    if (!ok && lane == 0) {
      const uint32_t from = issued > (uint32_t)p.stages ? issued - p.stages : 0u;
      for (uint32_t i = from; i < issued; ++i)
        mbar_wait_drain(b.full + 8 * (i % p.stages), (i / p.stages) & 1u, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_make(kBlk, kNT, false);
      int stage = 0, buf = 0, had = -1;
      uint32_t phase = 0, buf_phase = 0, h_phase = 0;
      bool any = false, ok = true;
      for (; w.more() && w.blk < nblk; w.next()) {
        if (w.blk != had) {  // this block's h is in tensor memory
          had = w.blk;
          ok = mbar_wait_one(b.done, h_phase, b.abort, p.status);
          h_phase ^= 1u;
        }
        ok = ok && mbar_wait_one(b.tempty + 8 * buf, buf_phase ^ 1u, b.abort, p.status) &&
             mbar_wait_one(b.full + 8 * stage, phase, b.abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sw = sbase + stage * p.stage_bytes;
        for (int part = 0; part < PARTS; ++part)
          for (int k = 0; k < p.rn / 16; ++k)
            tc_mma_ts(tmem + buf * kNT, h0 + part * hcols + k * 8,
                      sdesc_k_sw128(sw + (k >> 2) * kBoxBytes + (k & 3) * 32), idesc, part > 0 || k > 0);
        tc_commit(b.empty + 8 * stage);
        tc_commit(b.tfull + 8 * buf);
        any = true;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (!ok && any) {
        tc_commit(b.drain);
        mbar_wait_drain(b.drain, 0, 100000000ull);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3, group = (warp - 2) >> 2, half = group & 1, set = group >> 1;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t piece = sbase + p.base_off + (uint32_t)(half * 4 + q) * kPieceBytes;
    const uint32_t mine = (uint32_t)lane * kPieceRow;               // this thread's row of a piece
    const int sub = lane >> 3, chunk = lane & 7;                    // its place where 8 lanes share a row
    const int col = half * kHalf + chunk * (16 / (int)sizeof(T));  // column of its 16 bytes in a tile
    const uint32_t coal = (uint32_t)sub * kPieceRow + chunk * 16;
    const uint32_t row_bytes = (uint32_t)p.N * (uint32_t)sizeof(T);
    // the tokens of rows sub, sub + 4, ... of this warp, for the block that is loaded and the one that is stored
    auto tokens = [&](int blk, int (&tok)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = p.sorted[(size_t)blk * kBlk + q * 32 + sub + 4 * i];
        tok[i] = (unsigned)t < (unsigned)p.T ? t : -1;
      }
    };
    int ltok[8], stok[8];
    LoraWalk ld = w;
    if (set && ld.more()) ld.next();
    int lblk = -1, li = 0;
    auto load = [&]() {  // base of this set's next tile
      if (ld.more()) {
        const int n = ld.tile * kNT + col;
        if (p.base) {
          if (ld.blk != lblk) {
            lblk = ld.blk;
            tokens(lblk, ltok);
          }
          const uint32_t dst = piece + (uint32_t)(2 * li + set) * (8 * kPieceBytes) + coal;
          const char* src = static_cast<const char*>(p.base) + (size_t)n * sizeof(T);
          if (n < p.N) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (ltok[i] >= 0) cp_async16(dst + i * 4 * kPieceRow, src + (uint64_t)(uint32_t)ltok[i] * row_bytes, true);
          }
        }
        li ^= 1;
        ld.next();
        if (ld.more()) ld.next();
      }
      cp_async_commit();
    };
    load();
    // h of a block: pieces of 8 columns, every fourth to a group of warps; the first kHeld of the next block's are
    // fetched while this one is at work
    constexpr int kHeld = 4;
    const int pieces = PARTS * (p.rn / 8);
    uint4 held[kHeld];
    auto fetch = [&](int blk) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (group + 4 * u < pieces) held[u] = __ldcg(p.hp + ((size_t)blk * pieces + group + 4 * u) * kBlk + q * 32 + lane);
    };
    if (w.more() && w.blk < nblk) fetch(w.blk);
    const int last_blk = w.more() ? min(nblk - 1, (w.end - 1) / w.tiles) : 0;
    int had = -1, with_h = -1, si = 0;
    for (int i = 0; w.more(); ++i, w.next()) {
      const bool adapter = w.blk < nblk;
      if (w.blk != had) {
        had = w.blk;
        tokens(had, stok);
      }
      if (adapter && w.blk != with_h) {
        // (the products with the block before have to have ended)
        if (i && !__all_sync(0xffffffffu, mbar_wait_one(b.tfull + 8 * ((i - 1) & 1), ((i - 1) >> 1) & 1, b.abort, p.status)))
          break;
        tc_fence_after();  // (and the stores below come behind them)
        with_h = w.blk;
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
          if (group + 4 * u < pieces) tmem_st4(h0 + lanes + (group + 4 * u) * 4, held[u]);
        for (int x = group + 4 * kHeld; x < pieces; x += 4)
          tmem_st4(h0 + lanes + x * 4, __ldcg(p.hp + ((size_t)had * pieces + x) * kBlk + q * 32 + lane));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.done);
        if (had < last_blk) fetch(had + 1);
      }
      if ((i & 1) == set) {
        load();
        cp_async_wait<1>();
        __syncwarp();
        if (adapter) {
          if (!__all_sync(0xffffffffu, mbar_wait_one(b.tfull + 8 * set, (i >> 1) & 1, b.abort, p.status))) break;
          tc_fence_after();
        }
        const uint32_t at = piece + (uint32_t)(2 * si + set) * (8 * kPieceBytes);
        si ^= 1;
#pragma unroll
        for (int c = 0; c < kHalf; c += 32) {
          constexpr int kUnits = 32 * sizeof(T) / 16;
          uint32_t v[32];
          uint4 o[kUnits];
          if (adapter) {
            tmem_ld32_issue(tmem + set * kNT + lanes + half * kHalf + c, v);
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u) v[u] = 0;
          }
          const uint32_t sa = at + mine + c * (int)sizeof(T);
#pragma unroll
          for (int u = 0; u < kUnits; ++u) o[u] = p.base ? lds_v4(sa + u * 16) : make_uint4(0, 0, 0, 0);
          tmem_wait_ld();
          tmem_landed(v);
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            uint32_t* e = reinterpret_cast<uint32_t*>(&o[u]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if constexpr (sizeof(T) == 4)
                e[x] = __float_as_uint(__uint_as_float(e[x]) + __uint_as_float(v[4 * u + x]));
              else
                e[x] = pack_bf16x2(bf16_bits_to_f32(e[x] & 0xffffu) + __uint_as_float(v[8 * u + 2 * x]),
                                   bf16_bits_to_f32(e[x] >> 16) + __uint_as_float(v[8 * u + 2 * x + 1]));
            }
          }
#pragma unroll
          for (int u = 0; u < kUnits; ++u) sts_v4(sa + u * 16, o[u]);
        }
        tc_fence_before();
        __syncwarp();
        if (adapter && lane == 0) mbar_arrive(b.tempty + 8 * set);
        const int n = w.tile * kNT + col;
        if (n < p.N) {
          char* dst = static_cast<char*>(p.out) + (size_t)n * sizeof(T);
          uint4 o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = lds_v4(at + coal + e * 4 * kPieceRow);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (stok[e] >= 0) *reinterpret_cast<uint4*>(dst + (uint64_t)(uint32_t)stok[e] * row_bytes) = o[e];
        }
        __syncwarp();  // (the piece may be loaded again)
      }
    }
    cp_async_wait<0>();
  }
  tc_finish(b, tmem, kExpandCols);
}

// The tensor-core path's shape for a problem (from its sizes alone).
struct LoraPlan {
  bool tc;
  int rn, nblk, kb_total, kb_per, splits;
  long cap;
  size_t o_sorted, o_eids, o_meta, o_h, total;
};

LoraPlan lora_plan(int T, int K, int N, int r, int L) {
  LoraPlan q = {};
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  // Which path, by what each was measured to cost (us).  A token at a time: 5, and the adapters' rows of every
  // token at 9 TB/s (mostly from L2: with 16 adapters 512 tokens of rank 8 through 4096 x 4096 11.9, 256 of rank 64 35, 1024
  // of rank 16 41, 256 of rank 128 through 8192 x 8192 119).  Tensor cores: 13, every adapter's rows once from memory, and
  // 0.009 for each output tile of a block, however few its tokens (the same four: 19.9, 22, 21.3, 35).
  const long named = std::min(L, T), blocks = std::max(named, T / kBlk + named / 2 + 1);  // (as far as T and L tell)
  const double adapter = 2.0 * r * ((double)K + N);
  const double one_by_one = 5.0 + T * adapter / 9e6;
  const double sorted = 13.0 + named * adapter / 6.5e6 + 0.009 * blocks * ((N + 127) / 128);
  q.tc = one_by_one > sorted && N < (1 << 30);  // (the tensor-core kernels count a row's bytes in 32 bits)
  if (!q.tc) {
    q.total = up((size_t)T * r * sizeof(float));
    return q;
  }
  q.rn = (r + 15) / 16 * 16;
  q.cap = (long)T + (long)std::min(L + 1, T) * (kBlk - 1);  // (an adapter's tokens, and those without one, to whole blocks)
  q.nblk = (int)(q.cap / kBlk);
  q.kb_total = (K + 63) / 64;
  // a cluster shares a block's K where blocks are few: as many runs as keep all CTAs resident (a block to each
  // adapter, the last one of each half full on average), of 4 K blocks at least and none of them empty
  int n = 1;
  while (n < kMaxSplits && blocks * 2 * n <= kSlots && q.kb_total >= 8 * n) n *= 2;
  for (;; n /= 2) {
    q.kb_per = (q.kb_total + n - 1) / n;
    if (q.kb_per * (n - 1) < q.kb_total) break;
  }
  q.splits = n;
  q.o_sorted = 0;
  q.o_eids = up(q.cap * sizeof(int32_t));
  q.o_meta = q.o_eids + up((size_t)q.nblk * sizeof(int32_t));
  q.o_h = q.o_meta + up((size_t)meta_words(L + 1) * sizeof(int32_t));
  q.total = q.o_h + up((size_t)q.nblk * kBlk * q.rn * kMaxParts * 2);
  return q;
}

cudaError_t smem_limit(const void* kernel, bool (&set)[64], size_t bytes) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) set[dev] = true;
  return e;
}

constexpr size_t kSmemHalf = 112 * 1024;  // two CTAs to an SM
constexpr size_t kSmemMax = 227 * 1024;

template <typename T, int PARTS>
cudaError_t launch_expand(const LoraArgs& a, LoraTcDev p, cudaStream_t s) {
  constexpr int kNT = 2 * kSegBytes / sizeof(T);
  CUtensorMap tmB;
  if (!make_tensor_map_2d(&tmB, a.b, 2, a.r, (uint64_t)a.L * a.N, kNT)) return cudaErrorInvalidValue;
  p.stage_bytes = (uint32_t)((a.r + 63) / 64) * kNT * 128;
  const uint32_t base_bytes = kBaseStages * 8 * kPieceBytes;
  p.stages = std::min<int>(kMaxStages, (int)((kSmemMax - 1024 - kBarBytes - base_bytes) / p.stage_bytes));
  p.base_off = p.stages * p.stage_bytes;
  p.bar_off = p.base_off + base_bytes;
  p.n_tiles = (a.N + kNT - 1) / kNT;
  static bool set[64] = {};
  const cudaError_t e = smem_limit(reinterpret_cast<const void*>(k_lora_expand_tc<T, PARTS>), set, kSmemMax);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long>(a.num_sms, (long)p.nblk_max * p.n_tiles);
  MOE_LAUNCH((k_lora_expand_tc<T, PARTS>), dim3(grid), dim3(kExpandThreads), 1024 + p.bar_off + kBarBytes, s, tmB, p);
  return cudaGetLastError();
}

template <int STAGES>
cudaError_t launch_shrink(const CUtensorMap& tmA, LoraTcDev p, cudaStream_t s) {
  static bool set[64] = {};
  const cudaError_t e = smem_limit(reinterpret_cast<const void*>(k_lora_shrink_tc<STAGES>), set, kSmemHalf);
  if (e != cudaSuccess) return e;
  p.stage_bytes = kBlk * 128 + (uint32_t)p.rn * 128;
  p.bar_off = STAGES * p.stage_bytes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.nblk_max * p.splits);
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.dynamicSmemBytes = 1024 + p.bar_off + kBarBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_lora_shrink_tc<STAGES>, tmA, p);
}

cudaError_t launch_lora_tc(const LoraArgs& a, const LoraPlan& q, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + q.o_sorted);
  int32_t* eids = reinterpret_cast<int32_t*>(ws + q.o_eids);
  int32_t* meta = reinterpret_cast<int32_t*>(ws + q.o_meta);
  CUtensorMap tmA;
  if (!make_tensor_map_2d(&tmA, a.a, 2, a.K, (uint64_t)a.L * a.r, a.r)) return cudaErrorInvalidValue;
  cudaError_t e = launch_align(a.ids, a.T, 1, a.L + 1, kBlk, sorted, eids, meta + META_NPP, nullptr, meta, a.status, s, true,
                               nullptr, nullptr, 0, nullptr, INT32_MAX, true);
  if (e != cudaSuccess) return e;
  LoraTcDev p = {};
  p.T = a.T;
  p.K = a.K;
  p.N = a.N;
  p.r = a.r;
  p.L = a.L;
  p.rn = q.rn;
  p.nblk_max = q.nblk;
  p.kb_total = q.kb_total;
  p.kb_per = q.kb_per;
  p.splits = q.splits;
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.sorted = sorted;
  p.eids = eids;
  p.meta = meta;
  p.scale = a.scale;
  p.hp = reinterpret_cast<uint4*>(ws + q.o_h);
  p.parts = a.out_bf16 ? 2 : kMaxParts;
  p.base = a.base;
  p.out = a.out;
  p.status = a.status;
  e = q.rn <= 16   ? launch_shrink<6>(tmA, p, s)  // (as many stages as leave room for two CTAs)
      : q.rn <= 32 ? launch_shrink<5>(tmA, p, s)
      : q.rn <= 64 ? launch_shrink<4>(tmA, p, s)
                   : launch_shrink<3>(tmA, p, s);
  if (e != cudaSuccess) return e;
  return a.out_bf16 ? launch_expand<__nv_bfloat16, 2>(a, p, s) : launch_expand<float, kMaxParts>(a, p, s);
}

}  // namespace

size_t lora_workspace_bytes(int T, int K, int N, int r, int L) {
  return T == 0 ? 0 : lora_plan(T, K, N, r, L).total;
}

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) {
  const LoraPlan q = lora_plan(a.T, a.K, a.N, a.r, a.L);
  if (q.tc) return launch_lora_tc(a, q, s);
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
  return a.out_bf16 ? launch_few<__nv_bfloat16>(p, s) : launch_few<float>(p, s);
}

}  // namespace moe
