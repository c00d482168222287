// Low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + s[l] B_l (A_l x_t),  l = ids[t];  out[t] = base[t] where ids[t] = -1
//
// Few tokens: two launches on the CUDA cores, h = s A x (fp32, in the workspace), then out = base + B h, a
// token at a time (its adapter's rows come from L2 where tokens share them).
//
// More: the tokens are sorted by adapter (the permutation of the expert layer, an adapter in the place of an
// expert, blocks of 128 tokens), and both products run on the tensor cores, kind::f16 with fp32 sums:
//   shrink   a CTA to a block and a run of K: D[128 tokens x r] += X A^T over blocks of 64 K, both operands by
//            TMA (X as a box where the block's tokens are neighbours, else four rows to a gather); its fp32
//            sums go to the workspace, one plane for each run
//   expand   a CTA to a block and every R-th tile of 64 columns: h = s * (the planes' sum, in their order)
//            becomes the A operand in tensor memory, as bf16 parts that add up to it (2 for a bf16 output: off
//            by 2^-17 of h at most; 3 for an fp32 one: 2^-25), B's rows come by TMA, and the epilogue adds the base
// A token's row of D depends on that token alone, so what padding rows of a block hold does not matter.
// Two launches rather than clusters that exchange h: a CTA that holds tensor memory then never waits for
// another CTA.
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

// ---------------------------------------------------------------------------
// tensor cores
// ---------------------------------------------------------------------------
constexpr int kBlk = 128;          // tokens of a block
constexpr int kMaxStages = 6;
constexpr int kNT = 64;            // output columns of a tile
constexpr int kMaxBufs = 4;
constexpr int kShrinkThreads = 192;  // producer, MMA, 4 epilogue warps
constexpr int kExpandThreads = 320;  // producer, MMA, 8 epilogue warps

struct LoraTcDev {
  int T, K, N, r, L;
  int rn;                 // rank rounded up to 16
  int nblk_max;           // planes of the partial sums are this many blocks long
  int splits, kb_total, kb_per;
  int stages;
  uint32_t stage_bytes, bar_off;
  int parts, bufs, tmem_cols;
  int n_tiles, ranges;
  int wide;               // rows of base and out are whole 32-byte units
  int copy_ctas;          // grid columns behind the blocks that copy the rows without an adapter
  const int32_t *ids, *sorted, *eids, *meta;
  const float* scale;
  float* part;            // [splits][nblk_max][rn / 4][128] float4
  const void* base;
  void* out;
  int* status;
};

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
  b.tempty = b.tfull + 8 * kMaxBufs;
  b.done = b.tempty + 8 * kMaxBufs;
  b.drain = b.done + 8;
  b.exit = b.drain + 8;
  b.slot = reinterpret_cast<uint32_t*>(smem + off + 8 * (2 * kMaxStages + 2 * kMaxBufs + 3));
  b.abort = reinterpret_cast<volatile int*>(b.slot + 1);
  return b;
}
constexpr uint32_t kBarBytes = 8 * (2 * kMaxStages + 2 * kMaxBufs + 3) + 16;

// Barriers and tensor memory of a CTA; every thread.  done_count: arrivals of `done`.
__device__ __forceinline__ uint32_t tc_setup(const TcBars& b, const LoraTcDev& p, int cols, int done_count) {
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(b.full + 8 * s, 1);
      mbar_init(b.empty + 8 * s, 1);
    }
    for (int i = 0; i < kMaxBufs; ++i) {
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

__global__ void __launch_bounds__(kShrinkThreads)
    k_lora_shrink_tc(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmXg, const LoraTcDev p) {
  pdl_wait();
  const int blk = blockIdx.x, split = blockIdx.y;
  if (blk >= p.meta[META_NBLK]) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const TcBars b = tc_bars(smem, p.bar_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = pow2_cols(p.rn);
  const uint32_t tmem = tc_setup(b, p, cols, 1);
  // Dependents launch once the permutation is complete (this kernel's own wait) and every CTA here holds its
  // tensor memory: the expand kernel's CTAs take theirs before they wait for this kernel.
  pdl_launch_dependents();
  const int kb0 = split * p.kb_per, kb1 = min(kb0 + p.kb_per, p.kb_total);
  constexpr uint32_t kXBytes = kBlk * 128;

  if (warp == 0) {
    const int l = p.eids[blk];
    // the block's tokens, four to a lane; padding entries are T or more
    const int4 s4 = reinterpret_cast<const int4*>(p.sorted + (size_t)blk * kBlk)[lane];
    int row[4] = {s4.x, s4.y, s4.z, s4.w};
    int mine = 0;
    bool near = true;
    const int first = __shfl_sync(0xffffffffu, row[0], 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = (unsigned)row[i] < (unsigned)p.T;
      mine += in;
      near = near && (!in || row[i] == first + 4 * lane + i);
      if (!in) row[i] = row[0];
    }
    const int count = __reduce_add_sync(0xffffffffu, (unsigned)mine);
    // (a box reads 128 rows whatever their number: only where most of them are wanted)
    const bool box = __all_sync(0xffffffffu, near) && count > kBlk / 2;
    const uint32_t xbytes = box ? kXBytes : (uint32_t)((count + 3) / 4) * 512u;
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_all(b.empty + 8 * stage, phase ^ 1u, b.abort, p.status)) {
        ok = false;
        break;
      }
      const uint32_t sx = sbase + stage * p.stage_bytes, fb = b.full + 8 * stage;
      if (lane == 0) {
        mbar_arrive_expect_tx(fb, xbytes + (uint32_t)p.r * 128u);
        tma_load_2d(sx + kXBytes, &tmA, kb * 64, l * p.r, fb);
        if (box) tma_load_2d(sx, &tmX, kb * 64, first, fb);
      }
      __syncwarp();
      if (!box && 4 * lane < count)
        tma_gather4(sx + (uint32_t)lane * 512u, &tmXg, kb * 64, row[0], row[1], row[2], row[3], fb);
      __syncwarp();
      ++issued;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {  // let the copies already in flight land before the CTA exits
      const uint32_t from = issued > (uint32_t)p.stages ? issued - p.stages : 0u;
      for (uint32_t i = from; i < issued; ++i)
        mbar_wait_drain(b.full + 8 * (i % p.stages), (i / p.stages) & 1u, 100000000ull);
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
        if (++stage == p.stages) {
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
    const int q = warp & 3, row = q * 32 + lane;
    const bool ok = __all_sync(0xffffffffu, mbar_wait_one(b.done, 0, b.abort, p.status));
    tc_fence_after();
    if (ok) {
      float4* dst = reinterpret_cast<float4*>(p.part) + ((size_t)split * p.nblk_max + blk) * (p.rn / 4) * kBlk + row;
      for (int c = 0; c < p.rn; c += 16) {
        float v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[(size_t)(c / 4 + i) * kBlk] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
  }
  tc_finish(b, tmem, cols);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void ld_v8(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void st_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 columns of a row of base or out: UNITS times 32 bytes, those within the row
template <typename T>
struct RowPiece {
  static constexpr int kUnits = 32 * sizeof(T) / 32;
  static constexpr int kPer = 32 / sizeof(T);  // columns of a unit
  uint32_t v[kUnits][8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0;
  }
  __device__ __forceinline__ void load(const T* at, int left, bool wide) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (wide) {
        if (u * kPer < left) ld_v8(at + u * kPer, v[u]);
      } else {
        if (u * kPer < left) {
          const uint4 a = *reinterpret_cast<const uint4*>(at + u * kPer);
          v[u][0] = a.x; v[u][1] = a.y; v[u][2] = a.z; v[u][3] = a.w;
        }
        if (u * kPer + kPer / 2 < left) {
          const uint4 a = *reinterpret_cast<const uint4*>(at + u * kPer + kPer / 2);
          v[u][4] = a.x; v[u][5] = a.y; v[u][6] = a.z; v[u][7] = a.w;
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* at, int left, bool wide) const {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (wide) {
        if (u * kPer < left) st_v8(at + u * kPer, v[u]);
      } else {
        if (u * kPer < left) *reinterpret_cast<uint4*>(at + u * kPer) = make_uint4(v[u][0], v[u][1], v[u][2], v[u][3]);
        if (u * kPer + kPer / 2 < left)
          *reinterpret_cast<uint4*>(at + u * kPer + kPer / 2) = make_uint4(v[u][4], v[u][5], v[u][6], v[u][7]);
      }
    }
  }
  // this += f, each sum rounded once
  __device__ __forceinline__ void add(const uint32_t (&f)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i / 8][i % 8] = __float_as_uint(__uint_as_float(v[i / 8][i % 8]) + __uint_as_float(f[i]));
      } else if (i % 2 == 0) {
        uint32_t& w = v[i / 16][i % 16 / 2];
        w = pack_bf16x2(bf16_bits_to_f32(w & 0xffffu) + __uint_as_float(f[i]),
                        bf16_bits_to_f32(w >> 16) + __uint_as_float(f[i + 1]));
      }
    }
  }
};

template <typename T>
__device__ void lora_copy_rows(const LoraTcDev& p, int cta, int ctas) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int vecs = (int)((size_t)p.N * sizeof(T) / 16);
  for (int t = cta * warps + (threadIdx.x >> 5); t < p.T; t += ctas * warps) {
    const int l = p.ids[t];
    if (l >= 0 && l < p.L) continue;
    const uint4* src = static_cast<const uint4*>(p.base) + (size_t)t * vecs;
    uint4* dst = static_cast<uint4*>(p.out) + (size_t)t * vecs;
#pragma unroll 4
    for (int v = lane; v < vecs; v += 32) dst[v] = p.base ? src[v] : make_uint4(0, 0, 0, 0);
  }
}

template <typename T, int PARTS>
__global__ void __launch_bounds__(kExpandThreads)
    k_lora_expand_tc(const __grid_constant__ CUtensorMap tmB, const LoraTcDev p) {
  const int blk = blockIdx.x;
  if (blk >= p.nblk_max) {
    pdl_wait();
    pdl_launch_dependents();
    lora_copy_rows<T>(p, (blk - p.nblk_max) * gridDim.y + blockIdx.y, p.copy_ctas * gridDim.y);
    return;
  }
  // The permutation, base and the weights were complete before the preceding kernel let this one start; only
  // its sums are not.
  if (blk >= p.meta[META_NBLK]) {
    pdl_wait();
    return;
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const TcBars b = tc_bars(smem, p.bar_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = tc_setup(b, p, p.tmem_cols, 8);
  const uint32_t hcols = (uint32_t)(p.rn / 2);  // columns of one part of h
  const uint32_t d0 = tmem, h0 = tmem + (uint32_t)(p.bufs * kNT);
  const int l = p.eids[blk];
  const int kboxes = (p.r + 63) / 64;
  constexpr uint32_t kBoxBytes = kNT * 128;

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int j = blockIdx.y; j < p.n_tiles; j += p.ranges) {
      if (!mbar_wait_all(b.empty + 8 * stage, phase ^ 1u, b.abort, p.status)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        const uint32_t sw = sbase + stage * p.stage_bytes, fb = b.full + 8 * stage;
        mbar_arrive_expect_tx(fb, (uint32_t)kboxes * kBoxBytes);
        for (int x = 0; x < kboxes; ++x) tma_load_2d(sw + x * kBoxBytes, &tmB, x * 64, l * p.N + j * kNT, fb);
      }
      __syncwarp();
      ++issued;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    pdl_wait();
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
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool any = false;
      bool ok = mbar_wait_one(b.done, 0, b.abort, p.status);  // h is in tensor memory
      for (int j = blockIdx.y; j < p.n_tiles && ok; j += p.ranges) {
        ok = mbar_wait_one(b.tempty + 8 * buf, buf_phase ^ 1u, b.abort, p.status) &&
             mbar_wait_one(b.full + 8 * stage, phase, b.abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sw = sbase + stage * p.stage_bytes;
        for (int part = 0; part < PARTS; ++part)
          for (int k = 0; k < p.rn / 16; ++k)
            tc_mma_ts(d0 + buf * kNT, h0 + part * hcols + k * 8,
                      sdesc_k_sw128(sw + (k >> 2) * kBoxBytes + (k & 3) * 32), idesc, part > 0 || k > 0);
        tc_commit(b.empty + 8 * stage);
        tc_commit(b.tfull + 8 * buf);
        any = true;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == p.bufs) {
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
    const int q = warp & 3, half = (warp - 2) >> 2, row = q * 32 + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const int t = p.sorted[(size_t)blk * kBlk + row];
    const bool in = (unsigned)t < (unsigned)p.T;
    const T* base = p.base && in ? static_cast<const T*>(p.base) + (size_t)t * p.N : nullptr;
    T* out = in ? static_cast<T*>(p.out) + (size_t)t * p.N : nullptr;
    RowPiece<T> next;
    next.zero();
    auto fetch = [&](int j) {
      const int n = j * kNT + half * 32;
      if (base && j < p.n_tiles) next.load(base + n, p.N - n, p.wide);
    };
    fetch(blockIdx.y);
    const float s = p.scale ? p.scale[l] : 1.0f;
    pdl_wait();
    // h, 16 columns (one MMA step) at a time
    for (int c = half * 16; c < p.rn; c += 32) {
      float h[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = 0.f;
      const float4* src = reinterpret_cast<const float4*>(p.part) + ((size_t)blk * (p.rn / 4) + c / 4) * kBlk + row;
      for (int sp = 0; sp < p.splits; ++sp) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = src[((size_t)sp * p.nblk_max * (p.rn / 4) + i) * kBlk];
          h[4 * i] += v.x; h[4 * i + 1] += v.y; h[4 * i + 2] += v.z; h[4 * i + 3] += v.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = c + i < p.r ? h[i] * s : 0.f;
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = pack_bf16x2(h[2 * i], h[2 * i + 1]);
          h[2 * i] -= bf16_bits_to_f32(w[i] & 0xffffu);
          h[2 * i + 1] -= bf16_bits_to_f32(w[i] >> 16);
        }
        tmem_st8(h0 + lanes + part * hcols + c / 2, w);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(b.done);
    int buf = 0;
    uint32_t buf_phase = 0;
    for (int j = blockIdx.y; j < p.n_tiles; j += p.ranges) {
      RowPiece<T> cur = next;
      fetch(j + p.ranges);
      const bool ok = __all_sync(0xffffffffu, mbar_wait_one(b.tfull + 8 * buf, buf_phase, b.abort, p.status));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32_issue(d0 + buf * kNT + lanes + half * 32, v);
      tmem_wait_ld();
      tmem_landed(v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b.tempty + 8 * buf);
      if (++buf == p.bufs) {
        buf = 0;
        buf_phase ^= 1u;
      }
      cur.add(v);
      const int n = j * kNT + half * 32;
      if (out) cur.store(out + n, p.N - n, p.wide);
    }
  }
  tc_finish(b, tmem, p.tmem_cols);
}

// The tensor-core path's shape for a problem (from its sizes alone).
struct LoraPlan {
  bool tc;
  int rn, nblk, splits, kb_total, kb_per, ranges, n_tiles;
  long cap;
  size_t o_sorted, o_eids, o_meta, o_part, total;
};

constexpr int kSlots = 152 * 2;  // CTAs of either kernel that are resident together

LoraPlan lora_plan(int T, int K, int N, int r, int L) {
  LoraPlan q = {};
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  q.tc = T > 64;
  if (!q.tc) {
    q.total = up((size_t)T * r * sizeof(float));
    return q;
  }
  q.rn = (r + 15) / 16 * 16;
  q.cap = (long)T + (long)std::min(L, T) * (kBlk - 1);
  q.nblk = (int)(q.cap / kBlk);
  q.kb_total = (K + 63) / 64;
  const int want = std::max(1, std::min({kSlots / q.nblk, 8, q.kb_total / 4}));
  q.kb_per = (q.kb_total + want - 1) / want;
  q.splits = (q.kb_total + q.kb_per - 1) / q.kb_per;
  q.n_tiles = (N + kNT - 1) / kNT;
  q.ranges = std::max(1, std::min(q.n_tiles, (kSlots + q.nblk - 1) / q.nblk));
  q.o_sorted = 0;
  q.o_eids = up(q.cap * sizeof(int32_t));
  q.o_meta = q.o_eids + up((size_t)q.nblk * sizeof(int32_t));
  q.o_part = q.o_meta + up((size_t)meta_words(L) * sizeof(int32_t));
  q.total = q.o_part + up((size_t)q.splits * q.nblk * kBlk * q.rn * sizeof(float));
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

constexpr size_t kSmemMax = 112 * 1024;  // two CTAs to an SM

template <typename T, int PARTS>
cudaError_t launch_expand(const CUtensorMap& tmB, const LoraTcDev& p, dim3 grid, size_t smem, cudaStream_t s) {
  static bool set[64] = {};
  const cudaError_t e = smem_limit(reinterpret_cast<const void*>(k_lora_expand_tc<T, PARTS>), set, kSmemMax);
  if (e != cudaSuccess) return e;
  MOE_LAUNCH((k_lora_expand_tc<T, PARTS>), grid, dim3(kExpandThreads), smem, s, tmB, p);
  return cudaGetLastError();
}

cudaError_t launch_lora_tc(const LoraArgs& a, const LoraPlan& q, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  int32_t* sorted = reinterpret_cast<int32_t*>(ws + q.o_sorted);
  int32_t* eids = reinterpret_cast<int32_t*>(ws + q.o_eids);
  int32_t* meta = reinterpret_cast<int32_t*>(ws + q.o_meta);
  CUtensorMap tmA, tmX, tmXg, tmB;
  if (!make_tensor_map_2d(&tmA, a.a, 2, a.K, (uint64_t)a.L * a.r, a.r) ||
      !make_tensor_map_2d(&tmX, a.x, 2, a.K, a.T, kBlk) || !make_tensor_map_2d(&tmXg, a.x, 2, a.K, a.T, 1) ||
      !make_tensor_map_2d(&tmB, a.b, 2, a.r, (uint64_t)a.L * a.N, kNT))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_align(a.ids, a.T, 1, a.L, kBlk, sorted, eids, meta + META_NPP, nullptr, meta, a.status, s, true);
  if (e != cudaSuccess) return e;
  LoraTcDev p = {};
  p.T = a.T;
  p.K = a.K;
  p.N = a.N;
  p.r = a.r;
  p.L = a.L;
  p.rn = q.rn;
  p.nblk_max = q.nblk;
  p.splits = q.splits;
  p.kb_total = q.kb_total;
  p.kb_per = q.kb_per;
  p.n_tiles = q.n_tiles;
  p.ranges = q.ranges;
  p.ids = a.ids;
  p.sorted = sorted;
  p.eids = eids;
  p.meta = meta;
  p.scale = a.scale;
  p.part = reinterpret_cast<float*>(ws + q.o_part);
  p.base = a.base;
  p.out = a.out;
  p.status = a.status;
  {
    static bool set[64] = {};
    e = smem_limit(reinterpret_cast<const void*>(k_lora_shrink_tc), set, kSmemMax);
    if (e != cudaSuccess) return e;
    LoraTcDev d = p;
    d.stage_bytes = kBlk * 128 + (uint32_t)q.rn * 128;
    d.stages = std::min<int>(kMaxStages, (kSmemMax - 1024 - kBarBytes) / d.stage_bytes);
    d.bar_off = d.stages * d.stage_bytes;
    MOE_LAUNCH(k_lora_shrink_tc, dim3(q.nblk, q.splits), dim3(kShrinkThreads), 1024 + d.bar_off + kBarBytes, s, tmA, tmX,
               tmXg, d);
  }
  p.parts = a.out_bf16 ? 2 : 3;
  const int hcols = p.parts * q.rn / 2;
  p.tmem_cols = hcols + 2 * kNT <= 256 ? 256 : 512;
  p.bufs = std::min(kMaxBufs, (p.tmem_cols - hcols) / kNT);
  p.stage_bytes = (uint32_t)((a.r + 63) / 64) * kNT * 128;
  p.stages = kMaxStages;
  p.bar_off = p.stages * p.stage_bytes;
  const size_t row = (size_t)a.N * (a.out_bf16 ? 2 : 4);
  p.wide = row % 32 == 0 && (reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.base)) % 32 == 0;
  p.copy_ctas = a.base == a.out ? 0 : std::max(1, std::min(a.T / 80, 152) / q.ranges);
  const dim3 grid(q.nblk + p.copy_ctas, q.ranges);
  const size_t smem = 1024 + p.bar_off + kBarBytes;
  return a.out_bf16 ? launch_expand<__nv_bfloat16, 2>(tmB, p, grid, smem, s) : launch_expand<float, 3>(tmB, p, grid, smem, s);
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
  const int rows = std::min(a.T, 1 << 16), cols = (a.N + 255) / 256;
  if (cols > 65535) return cudaErrorInvalidValue;
  MOE_LAUNCH(k_lora_shrink, dim3(rows, (a.r + 7) / 8), dim3(256), 0, s, p);
  if (a.out_bf16) MOE_LAUNCH(k_lora_expand<__nv_bfloat16>, dim3(rows, cols), dim3(256), 0, s, p);
  else MOE_LAUNCH(k_lora_expand<float>, dim3(rows, cols), dim3(256), 0, s, p);
  return cudaGetLastError();
}

}  // namespace moe
