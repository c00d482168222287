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
// Roles (320 threads): warp 0 streams operands by TMA into a ring of shared-memory stages, warp 1
// issues the MMAs into a ring of tensor-memory blocks, warps 2-9 fold the blocks (four
// of them D0, four D1: with four for both, a block of 64 tokens took 0.6 us, longer than its load).  Every wait is
// bounded; after one gives up, each role runs on without waiting or storing, so the barriers
// between the epilogue warps stay matched and the kernel ends.
//
// Few tiles (small batches): a cluster of 2, 4 or 8 CTAs shares a tile, each taking a run of its K
// blocks.  The sums meet in distributed shared memory -- every token's row is added up in rank order
// by one warp of one of the CTAs -- so there is no workspace, no second kernel and no order that
// changes between calls.
//
// Bound by HBM: 16 tokens x 8192 x 4096 7.8 us (4.4 TB/s with the launch), 16 tokens through 64 experts of
// 4096 x 8192 869 us (6.5 TB/s).
#include <algorithm>

#include "moe_align.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBgThreads = 320;  // 2 warps of roles, 8 epilogue warps
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
  int stages, out_bf16;
  int cl;               // CTAs of a cluster that share a tile's K blocks (1, 2, 4, 8)
  int kb_per;           // K blocks of one of them
  int early;            // the tile list and the weights may be read before the dependency wait
  int out_tma;          // CTA pairs: rows of out are whole 16-byte units
  int out_rows;         // rows of out
  uint32_t stage_bytes, bar_off, scale_off, out_off, list_off;
  const float* a_scale;  // [rows][kb_total]
  const float* w_scale;  // [E][w_scale_rows][kb_total]
  const int32_t* sorted;
  const int32_t* eids;
  const int32_t* meta;
  const int32_t* pblk;   // CTA pairs: the permutation's 256- and 128-row chunks
  const int32_t* ids;    // nullable: the routing itself instead of eids and meta (BlockGemmArgs)
  void* out;
  float* out_scale;
  int* status;
};

struct BgTile {
  int e, n, xrow, ntok, npad, wr0;
};

// Tiles of a routing of at most 32 pairs, in shared memory: expert and tokens of each permutation block.
struct BgList {
  int2 blk[kAlignSmallPairs];
  int n;
};

template <int NT>
__device__ __forceinline__ void bg_make_list(const BgDev& p, BgList* list) {  // (one warp)
  const SmallGroup g = align_small(p.ids, p.T * p.k, p.E, NT, nullptr, 1);
  if (g.leader)
    for (int b = 0; b < g.pad / NT; ++b) list->blk[g.off / NT + b] = make_int2(g.e, min(NT, g.count - b * NT));
  const int blocks = __reduce_add_sync(0xffffffffu, g.leader ? g.pad / NT : 0);
  if ((threadIdx.x & 31) == 0) list->n = blocks;
}

template <int EPI, int NT>
__device__ __forceinline__ int bg_tile_count(const BgDev& p, const BgList* list) {
  if constexpr (EPI == BG_EPI_DENSE) return (p.T + NT - 1) / NT * p.n_tiles;
  if constexpr (EPI == BG_EPI_G1)
    if (p.ids) return list->n * p.n_tiles;
  return p.meta[META_NBLK] * p.n_tiles;
}

template <int EPI, int NT>
__device__ __forceinline__ BgTile bg_tile_at(const BgDev& p, const BgList* list, int t) {
  BgTile d;
  const int m = t / p.n_tiles;
  d.n = t - m * p.n_tiles;
  d.xrow = m * NT;
  if constexpr (EPI == BG_EPI_DENSE) {
    d.e = 0;
    d.ntok = min(NT, p.T - d.xrow);
  } else if (EPI == BG_EPI_G1 && p.ids) {
    const int2 b = list->blk[m];
    d.e = b.x;
    d.ntok = b.y;
  } else {  // one block of the permutation (an expert's are neighbours: its weights come from L2 after the first)
    d.e = p.eids[m];
    d.ntok = min(NT, p.meta[meta_offsets(p.E) + d.e] + p.meta[meta_counts(p.E) + d.e] - d.xrow);
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

// One token's 256 sums by one warp: v0 columns 4 * lane.. of the tile's first 128 weight rows, v1 of
// the second.
template <int EPI>
__device__ __forceinline__ void bg_store_row(const BgDev& p, const BgTile& d, const float4& v0, const float4& v1, int c,
                                             int lane) {
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
    const size_t o = (size_t)f * p.n_out + (size_t)d.n * 256 + 4 * lane;
    const bool second = d.n * 256 + 128 < p.n_out;
    if (p.out_bf16) {  // (as k_gemm_block_pair)
      uint2* y = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + o);
      y[0] = make_uint2(pack_bf16x2(v0.x, v0.y), pack_bf16x2(v0.z, v0.w));
      if (second) y[32] = make_uint2(pack_bf16x2(v1.x, v1.y), pack_bf16x2(v1.z, v1.w));
    } else {
      float* y = static_cast<float*>(p.out) + o;
      *reinterpret_cast<float4*>(y) = v0;
      if (second) *reinterpret_cast<float4*>(y + 128) = v1;
    }
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
  constexpr int kPass = NT < kStageTokens ? NT : kStageTokens;  // tokens transposed at a time

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < kBgBufs; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, 8);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_exit, kBgThreads / 32);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kCols);
  BgList* list = reinterpret_cast<BgList*>(smem + p.list_off);
  if constexpr (EPI == BG_EPI_G1)
    if (p.ids && warp == 2) bg_make_list<NT>(p, list);
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // this CTA's share of a tile's K blocks, and its first tile (clusters: its only one)
  const int rank = p.cl > 1 ? (int)cluster_ctarank() : 0;
  const int kb0 = rank * p.kb_per, kb1 = min(kb0 + p.kb_per, p.kb_total);
  const int tile0 = blockIdx.x / p.cl, stride = gridDim.x / p.cl;
  if (!p.early) pdl_wait();
  const int ntiles = bg_tile_count<EPI, NT>(p, list);

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    int pre = 0;  // stages whose weights are already on their way
    if (p.early && tile0 < ntiles) {
      const BgTile d = bg_tile_at<EPI, NT>(p, list, tile0);
      pre = min(p.stages, kb1 - kb0);
      if (elect_one())
        for (int i = 0; i < pre; ++i) {
          const uint32_t sw = sbase + i * p.stage_bytes, fb = bar_full + 8 * i;
          mbar_arrive_expect_tx(fb, 2 * kHalfBytes + (uint32_t)d.npad * 128u);
          tma_load_2d(sw, &tmW, (kb0 + i) * 128, d.wr0, fb);
          tma_load_2d(sw + kHalfBytes, &tmW, (kb0 + i) * 128, d.wr0 + p.w_pair_off, fb);
        }
      __syncwarp();
    }
    if (p.early) pdl_wait();
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int t = tile0; t < ntiles && ok; t += stride) {
      const BgTile d = bg_tile_at<EPI, NT>(p, list, t);
      for (int kb = kb0; kb < kb1; ++kb) {
        const bool weights = (int)issued >= pre;
        if (weights && !mbar_wait_all(bar_empty + 8 * stage, phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sw = sbase + stage * p.stage_bytes, fb = bar_full + 8 * stage;
          if (weights) {
            mbar_arrive_expect_tx(fb, 2 * kHalfBytes + (uint32_t)d.npad * 128u);
            tma_load_2d(sw, &tmW, kb * 128, d.wr0, fb);
            tma_load_2d(sw + kHalfBytes, &tmW, kb * 128, d.wr0 + p.w_pair_off, fb);
          }
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
    // ---------------- MMA issuer: one thread ----------------
    if (p.early) pdl_wait();
    if (elect_one()) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true, any = false;
      for (int t = tile0; t < ntiles && ok; t += stride) {
        const uint32_t idesc = idesc_make(128, bg_tile_at<EPI, NT>(p, list, t).npad, true);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait_one(bar_tempty + 8 * buf, buf_phase ^ 1u, abort_flag, p.status) &&
               mbar_wait_one(bar_full + 8 * stage, phase, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
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
        tc_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0, 100000000ull);
      }
    }
    __syncwarp();
  }
  if (warp < 2) {
    if (p.cl > 1 && tile0 < ntiles) {  // the epilogue's cluster barriers take every thread
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    // ---------------- epilogue (warps 2..9): fold the blocks, then the outputs ----------------
    if (p.early) pdl_wait();
    const int q = warp & 3;          // tensor-memory lane quadrant this warp may read
    const int w8 = warp - 2, h = w8 >> 2;  // this warp's accumulator: D0 or D1
    const int lrow = q * 32 + lane;        // weight row of this thread in it
    const int tid = (threadIdx.x - 64) & 127;
    float* sc = reinterpret_cast<float*>(smem + p.scale_off);  // [2][2][kScaleChunk][NT]
    constexpr int kSet = kScaleChunk * NT;                     // scale products of one chunk and half
    constexpr int kPer = kSet / 128;
    const int lane_kb = tid % kScaleChunk, lane_c = tid / kScaleChunk;  // this thread's first scale of a chunk
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    for (int t = tile0; t < ntiles; t += stride) {
      const BgTile d = bg_tile_at<EPI, NT>(p, list, t);
      const int srow = d.n * (p.w_tile_rows / 128);
      const float* ws = p.w_scale + ((size_t)d.e * p.w_scale_rows +
                                     min(srow + h * p.s_pair_off, p.w_scale_rows - 1)) * p.kb_total;
      // scales of the next chunk, one K block and every 16th token to a thread
      float ra[kPer], rw = 0.0f;
      auto fetch = [&](int kb) {
        const bool in = kb + lane_kb < kb1;
        rw = in ? ws[kb + lane_kb] : 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = lane_c + i * (128 / kScaleChunk);
          ra[i] = (in && c < d.ntok) ? p.a_scale[(size_t)(d.xrow + c) * p.kb_total + kb + lane_kb] : 0.0f;
        }
      };
      float2 acc[NT / 2];
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      fetch(kb0);
      for (int kc = kb0, par = 0; kc < kb1; kc += kScaleChunk, par ^= 1) {
        float* sp = sc + (par * 2 + h) * kSet;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = lane_c + i * (128 / kScaleChunk);
          sp[lane_kb * NT + c] = ra[i] * rw;
        }
        named_bar_sync(1, 256);
        if (kc + kScaleChunk < kb1) fetch(kc + kScaleChunk);
        const int kn = min(kScaleChunk, kb1 - kc);
        for (int kb = 0; kb < kn; ++kb) {
          if (ok) ok = mbar_wait_one(bar_tfull + 8 * buf, buf_phase, abort_flag, p.status);
          __syncwarp();
          tc_fence_after();
          const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)((buf * 2 + h) * NT);
          constexpr int W = NT < 32 ? 16 : 32;  // columns of one load
#pragma unroll
          for (int c0 = 0; c0 < NT; c0 += W) {
            if (c0 < d.npad) {
              uint32_t v[W];
              tmem_ld_issue<W>(tb + c0, v);
              tmem_wait_ld();
              tmem_landed(v);
#pragma unroll
              for (int j = 0; j < W; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(sp + kb * NT + c0 + j);
                const int i = (c0 + j) / 2;
                fma2(acc[i], f.x, f.y, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                fma2(acc[i + 1], f.z, f.w, __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_tempty + 8 * buf);
          if (++buf == kBgBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      // A wait that gives up does so for each lane by itself.  The stores below shuffle over whole warps, so
      // a warp stores only if all of its lanes saw every block, and a token's row is stored by one warp.
      ok = __all_sync(0xffffffffu, ok);
      // transpose through shared memory: thread = weight row -> warp = token
      auto stage_tokens = [&](float* rows, int i0, int n) {  // (i0, n compile-time after unrolling)
#pragma unroll
        for (int c = 0; c < n; c += 2) {
          rows[c * 256 + 128 * h + lrow] = acc[i0 + c / 2].x;
          rows[(c + 1) * 256 + 128 * h + lrow] = acc[i0 + c / 2].y;
        }
      };
      if (p.cl == 1) {
        float* st = reinterpret_cast<float*>(smem + p.out_off);  // [kPass][256]
#pragma unroll
        for (int c0 = 0; c0 < NT; c0 += kPass) {
          if (c0 < d.ntok) {
            stage_tokens(st, c0 / 2, kPass);
            named_bar_sync(1, 256);
            if (ok)
              for (int c = w8; c < min(d.ntok - c0, kPass); c += 8) {
                const float4* row = reinterpret_cast<const float4*>(st + c * 256) + lane;
                bg_store_row<EPI>(p, d, row[0], row[32], c0 + c, lane);
              }
            named_bar_sync(1, 256);
          }
        }
      } else {
        // The ring is idle once the tile's last block has been folded (one tile to a CTA): it takes all
        // tokens' sums at once.  Rank r of the cluster stores tokens r, r + cl, ..., each added up in rank
        // order.
        stage_tokens(reinterpret_cast<float*>(smem), 0, NT);
        __syncwarp();
        cluster_sync_all();
        if (ok)
          for (int c = rank + w8 * p.cl; c < d.ntok; c += 8 * p.cl) {
            const uint32_t at = sbase + (uint32_t)(c * 256 + 4 * lane) * 4u;
            float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
            for (int r = 0; r < p.cl; ++r) {
              const uint32_t from = mapa_shared(at, r);
              const float4 a0 = ld_cluster_f32x4(from), a1 = ld_cluster_f32x4(from + 512u);
              v0.x += a0.x; v0.y += a0.y; v0.z += a0.z; v0.w += a0.w;
              v1.x += a1.x; v1.y += a1.y; v1.z += a1.z; v1.w += a1.w;
            }
            bg_store_row<EPI>(p, d, v0, v1, c, lane);
          }
        __syncwarp();
        cluster_sync_all();  // (no CTA leaves while another reads its rows)
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

// Smallest share of a tile's K blocks that a CTA of a cluster is given (below that its prologue and
// the exchange cost more than its share).
constexpr int kMinSplitBlocks = 3;

template <int EPI, int NT>
cudaError_t launch_bg(const CUtensorMap& mw, const CUtensorMap& mx, BgDev p, long tiles, int sms, cudaStream_t s) {
  p.stage_bytes = 2u * 128u * 128u + (uint32_t)NT * 128u;
  const uint32_t list_at = 8 * (2 * kBgMaxStages + 2 * kBgBufs + 2) + 16;  // behind the barriers and words
  const uint32_t bar_bytes = list_at + (uint32_t)sizeof(BgList);
  const uint32_t scale_bytes = 2u * 2u * kScaleChunk * NT * 4u;
  const uint32_t out_bytes = (uint32_t)std::min(NT, kStageTokens) * 256u * 4u;
  p.stages = std::min<int>(kBgMaxStages, (227 * 1024 - 1024 - bar_bytes - scale_bytes - out_bytes) / p.stage_bytes);
  p.out_off = (uint32_t)p.stages * p.stage_bytes;
  p.scale_off = p.out_off + out_bytes;
  p.bar_off = p.scale_off + scale_bytes;
  p.list_off = p.bar_off + list_at;
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
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kBgThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // CTAs that share one tile: as many as keep all tiles resident together (152 SMs hold 76 clusters
  // of 2, 36 of 4, 15 of 8: a sixteenth cluster of 8 would double the time)
  static int resident[4][64] = {};
  p.cl = 1;
  for (int i = 1; i < 4; ++i) {
    const int cl = 1 << i;
    if (p.kb_total / cl < kMinSplitBlocks || tiles * cl > sms) break;
    if (dev < 0 || dev >= 64) break;
    if (resident[i][dev] == 0) {
      attr[0].val.clusterDim.x = cl;
      cfg.gridDim = dim3(cl);
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = -1;
      }
      resident[i][dev] = n;
    }
    if (tiles > resident[i][dev]) break;
    p.cl = cl;
  }
  p.kb_per = (p.kb_total + p.cl - 1) / p.cl;
  // one tile to a CTA with clusters, a persistent grid without
  cfg.gridDim = dim3((unsigned)(p.cl > 1 ? tiles * p.cl : std::max<long>(1, std::min<long>(tiles, sms))));
  attr[0].val.clusterDim.x = p.cl;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, p);
}

template <int EPI>
cudaError_t launch_bg_nt(const CUtensorMap& mw, const CUtensorMap& mx, const BgDev& p, int nt, long tiles, int sms,
                         cudaStream_t s) {
  if (nt == 16) return launch_bg<EPI, 16>(mw, mx, p, tiles, sms, s);
  if (nt == 32) return launch_bg<EPI, 32>(mw, mx, p, tiles, sms, s);
  if (nt == 64) return launch_bg<EPI, 64>(mw, mx, p, tiles, sms, s);
  return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// Token-major products on CTA pairs (tcgen05 cta_group::2)
// ---------------------------------------------------------------------------
// A cluster of two CTAs computes 256 token rows x 256 weight rows; CTA r stages token rows
// [128r, 128r + 128) and weight box r (GEMM1: 128 gate rows, the matching 128 up rows).  Half j of a
// K block is one set of M = 256, N = 128 MMAs over rows [64j, 64j + 64) of both weight boxes, issued
// by CTA 0, and leaves each CTA 128 rows x (64 sums of box 0, 64 of box 1) in its tensor memory.
// The last tile of an expert (or of the batch) runs as M = 128 when it has at most 128 rows: CTA r
// then stages 64 of them, and lane i of its tensor memory holds row 64r + (i mod 64) and the 64 sums
// of box i / 64; for GEMM1 the boxes of such a tile interleave 32 gate and 32 up rows, so that gate
// and up of a column still meet in one thread.
//
// The fold is the work beside the MMAs: 128 x 256 sums per SM and K block, one packed fma for two of
// them.  Eight warps hold the 128 x 256 fp32 accumulators, 128 to a thread; four of them fold half 0,
// four half 1.  A sum can be overwritten only after its fold, and tensor memory holds two K blocks of
// the tile, so what limits the rate is the round trip MMA -> commit -> fold -> release -> MMA.  Halves
// cut it into four buffers instead of two: one is filled while three travel (N = 128 reads the token
// rows from shared memory twice, which costs less than waiting).
//
// 8192 x 4096 x 4096: 111 us, 2470 TFLOP/s (86 us without the fold, power-capped).  An expert layer of 8192
// tokens (64 experts, 4096 x 2048, top-8): GEMM1 990 us, GEMM2 500 us.
constexpr int kBpThreads = 384;                 // 4 warps of roles, 8 epilogue warps
constexpr int kBpRoleRegs = 72, kBpEpiRegs = 216;  // 72 + 2 * 216 = 3 * 168, the launch's registers
constexpr int kBpStages = 5;                    // (as fast as 6; the rows on their way out take the room)
constexpr uint32_t kBpHalf = 128u * 128u;       // bytes of a 128-row box of one K block
constexpr uint32_t kBpStage = 2u * kBpHalf;     // this CTA's weight box and token rows
constexpr uint32_t kBpOut = kBpStages * kBpStage;   // [8 warps][32 rows][128 bytes] output rows on their way
constexpr uint32_t kBpOutWarp = 32 * 128;
constexpr uint32_t kBpRed = kBpOut + 8 * kBpOutWarp;  // [2][256] block maxima of the epilogue halves
constexpr int kBpChunk = 4;                     // K blocks of one scale chunk
constexpr int kBpChunks = 4;                    // scale chunks in the ring (a power of two)
constexpr uint32_t kBpScale = kBpRed + 2 * 256 * 4;  // [chunk][block][128 rows] (scale of run a, of run b)
constexpr uint32_t kBpBar = kBpScale + kBpChunks * kBpChunk * 128 * 8;
// barriers and words behind them, from kBpBar: full, empty [stage]; tfull, tempty [buffer][half];
// drain [half]; sfull, sempty [chunk]; tensor-memory address, abort flag
constexpr uint32_t kBpTfull = 8 * 2 * kBpStages, kBpTempty = kBpTfull + 32, kBpDrain = kBpTempty + 32,
                   kBpSfull = kBpDrain + 16, kBpSempty = kBpSfull + 8 * kBpChunks,
                   kBpWords = kBpSempty + 8 * kBpChunks;
constexpr uint32_t kBpSmem = 1024 + kBpBar + kBpWords + 16;

struct BpTile {
  int e, n, xrow, wr0;
  bool tail;
};

template <int EPI>
__device__ __forceinline__ BpTile bp_tile_at(const BgDev& p, int t) {
  BpTile d;
  const int c = t / p.n_tiles;
  d.n = t - c * p.n_tiles;
  if constexpr (EPI == BG_EPI_DENSE) {
    d.e = 0;
    d.xrow = 256 * c;
    d.tail = p.T - d.xrow <= 128;
  } else {
    const int v = p.pblk[c];
    d.xrow = v >> 1;
    d.tail = (v & 1) != 0;
    d.e = p.eids[d.xrow / 128];
  }
  d.wr0 = d.e * p.w_rows + d.n * p.w_tile_rows;
  return d;
}

// acc[0..31] += s * (32 loaded sums)
__device__ __forceinline__ void bp_fold32(float2* acc, const uint32_t (&r)[32], float s) {
#pragma unroll
  for (int j = 0; j < 16; ++j) fma2(acc[j], s, s, __uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}

// SiLU(g) * u for an intermediate that becomes e4m3 (4 significant bits) right away.  The quotient is within 2
// ulp, the exponential within 2 + floor(1.173 |g|) (CUDA's bounds), and for a negative gate e^-g is the whole
// denominator: about 2^-22 relative near 0, 25 ulp (2^-18.4) at g = -20, 95 ulp (2^-16.4) at -80, and 0 below
// about -87.  Of the 25 million codes of 4096 tokens through 8 of 128 experts (2048 x 768) 14 differ from the
// rounded forms'.  64 of these per thread stand between two tiles: with the rounded quotient that layer takes
// 402 us instead of 275 and 8192 tokens through 64 experts of 4096 x 2048 1866 instead of 1628, with the
// rounded exponential alone 280 and 1647.
__device__ __forceinline__ float silu_mul_fast(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// 32 bytes, 32-byte aligned, in one store
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A warp's 32 rows (one to a lane) x 128 bytes from column col on, through shared memory by one TMA store:
// get(i) is columns 2i and 2i + 1 of the lane's row from there.  A lane's own stores, a row each, reach 32
// lines whatever their width, and until they were out the next tile's folds waited: with 32-byte stores
// 8192 x 4096 x 4096 took 119.5 us (this way 111), an expert GEMM2 of 65536 rows 577 us (500); a second
// buffer for a stage of the ring gains 1 % there and loses 4 % where weights are streamed.  Rows and columns
// past the end of out are clipped by the tensor map.
template <bool BF16, class Get>
__device__ __forceinline__ void bp_store_box(const BgDev& p, const CUtensorMap* tm, uint32_t buf, int lane, int row0,
                                             int col, Get get) {
  if (row0 >= p.out_rows || col >= p.n_out) return;  // (the same for the whole warp)
  if (lane == 0) bulk_wait_read();  // the rows stored before have left the buffer
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint4 v;
    if constexpr (BF16) {
      v = make_uint4(pack_bf16x2(get(4 * c).x, get(4 * c).y), pack_bf16x2(get(4 * c + 1).x, get(4 * c + 1).y),
                     pack_bf16x2(get(4 * c + 2).x, get(4 * c + 2).y), pack_bf16x2(get(4 * c + 3).x, get(4 * c + 3).y));
    } else {
      v = make_uint4(__float_as_uint(get(2 * c).x), __float_as_uint(get(2 * c).y), __float_as_uint(get(2 * c + 1).x),
                     __float_as_uint(get(2 * c + 1).y));
    }
    sts_v4(buf + lane * 128u + (uint32_t)((c ^ (lane & 7)) << 4), v);  // (the map's 128-byte swizzle)
  }
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tm, buf, BF16 ? col : 2 * col, row0);  // (fp32 rows as pairs of 16-bit elements)
    bulk_commit();
  }
}

// A thread's 2 * PAIRS consecutive output columns from column n of one row that is no whole 16-byte units.
template <int PAIRS>
__device__ __forceinline__ void bp_store(const BgDev& p, size_t row, int n, const float2* acc) {
  const size_t o = row * (size_t)p.n_out + n;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    const float v[2] = {acc[i].x, acc[i].y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (n + 2 * i + h >= p.n_out) continue;
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[o + 2 * i + h] = __float2bfloat16_rn(v[h]);
      else
        static_cast<float*>(p.out)[o + 2 * i + h] = v[h];
    }
  }
}

// What a thread keeps for the folds beside its accumulators.  Registers are short (128 sums, 64 loaded
// columns): a spilled word in the loop costs a tenth of the rate.  What the compiler does spill (20 bytes)
// stays out of it: 8192 x 4096 x 4096 executes 4 local loads per warp and tile, not one per K block.
struct BpFold {
  uint32_t bars;    // barriers of this CTA (kBpBar)
  uint32_t tmem;    // tensor-memory address of its half in buffer 0 (buffer 1: + 256 columns)
  uint32_t tfull;   // arrival barrier of its half in buffer 0 (buffer 1: + 16)
  uint32_t tempty;  // release barrier of its half in buffer 0 (buffer 1: + 16), in CTA 0
  uint32_t scale;   // this row's scale pair of block 0 of chunk 0
  uint32_t blocks;  // blocks folded so far: buffer and phase
  uint32_t chunks;  // scale chunks used so far
  bool ok;          // (per lane: a lane whose wait gave up goes on without waiting, and stores nothing)
};

__device__ __forceinline__ bool bp_wait(const BpFold& f, uint32_t bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int* abort_flag = static_cast<volatile int*>(__cvta_shared_to_generic(f.bars + kBpWords + 4));
  return mbar_wait_one(bar, parity, abort_flag, status);
}

__device__ __forceinline__ void bp_arrived(BpFold& f, int* status) {
  if (f.ok) f.ok = bp_wait(f, f.tfull + 16 * (f.blocks & 1u), (f.blocks >> 1) & 1u, status);
  __syncwarp();
  tc_fence_after();
}

__device__ __forceinline__ void bp_release(BpFold& f) {
  tc_fence_before();
  __syncwarp();
  if (elect_one()) mbar_arrive_remote(f.tempty + 16 * (f.blocks & 1u));  // (CTA 0's own included)
  ++f.blocks;
}

// All K blocks of a tile into acca / accb.  One chain of loads of 32 columns runs through the whole
// tile, also across blocks: while a chunk is folded the next one is on its way, and a block is
// released, and the next one's arrival awaited, before its last chunk is folded.  (Waiting, fences and
// loads one after another took about 1100 cycles a block; the MMAs of a block take about 600.)
template <bool TAIL>
__device__ __forceinline__ void bp_fold_tile(BpFold& f, int nkb, int* status, float2 (&acca)[32],
                                             float2 (&accb)[32]) {
  uint32_t r0[32], r1[32];
  bp_arrived(f, status);
  tmem_ld32_issue(f.tmem + 256 * (f.blocks & 1u), r0);
#pragma unroll 1
  for (int kb = 0; kb < nkb; ++kb) {
    const uint32_t slot = f.chunks & (kBpChunks - 1), i = kb & (kBpChunk - 1);
    if (i == 0) {
      if (f.ok) f.ok = bp_wait(f, f.bars + kBpSfull + 8 * slot, (f.chunks / kBpChunks) & 1u, status);
      __syncwarp();
    }
    const float2 s = lds_f32x2(f.scale + (slot * kBpChunk + i) * (128u * 8u));
    if (i == kBpChunk - 1 || kb == nkb - 1) {  // the chunk's last block: its scales are in registers
      __syncwarp();
      if (elect_one()) mbar_arrive(f.bars + kBpSempty + 8 * slot);
      ++f.chunks;
    }
    const uint32_t tb = f.tmem + 256 * (f.blocks & 1u);
    tmem_wait_ld();
    tmem_landed(r0);
    tmem_ld32_issue(tb + 32, r1);
    bp_fold32(acca, r0, s.x);
    if constexpr (!TAIL) {
      tmem_wait_ld();
      tmem_landed(r1);
      tmem_ld32_issue(tb + 64, r0);
      bp_fold32(acca + 16, r1, s.x);
      tmem_wait_ld();
      tmem_landed(r0);
      tmem_ld32_issue(tb + 96, r1);
      bp_fold32(accb, r0, s.y);
    }
    tmem_wait_ld();
    tmem_landed(r1);
    bp_release(f);
    if (kb + 1 < nkb) {
      bp_arrived(f, status);
      tmem_ld32_issue(f.tmem + 256 * (f.blocks & 1u), r0);
    }
    bp_fold32(TAIL ? accb : accb + 16, r1, s.y);
  }
}

// The rows and scales of a tile as tensor-memory lane `lrow` sees them.
template <int EPI>
__device__ __forceinline__ int bp_row(const BpTile& d, uint32_t rank, int lrow) {
  return d.xrow + (d.tail ? 64 * (int)rank + (lrow & 63) : 128 * (int)rank + lrow);
}
template <int EPI>
__device__ __forceinline__ void bp_scale_rows(const BgDev& p, const BpTile& d, int lrow, const float*& wsa,
                                              const float*& wsb) {
  constexpr bool G1 = EPI == BG_EPI_G1;
  const int hf = d.tail ? lrow >> 6 : 0, last = p.w_scale_rows - 1;
  const int ra = G1 ? d.n : min(2 * d.n + hf, last);
  const int rb = G1 ? d.n + p.s_pair_off : d.tail ? ra : min(2 * d.n + 1, last);
  wsa = p.w_scale + ((size_t)d.e * p.w_scale_rows + ra) * p.kb_total;
  wsb = p.w_scale + ((size_t)d.e * p.w_scale_rows + rb) * p.kb_total;
}

template <int EPI>
__global__ void __launch_bounds__(kBpThreads, 1)
    k_gemm_block_pair(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ CUtensorMap tmW32, const __grid_constant__ CUtensorMap tmX64,
                      const __grid_constant__ CUtensorMap tmO, const BgDev p) {
  constexpr bool G1 = EPI == BG_EPI_G1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + kBpBar;
  const uint32_t bar_empty = bar_full + 8 * kBpStages;
  const uint32_t bar_tfull = bar_full + kBpTfull;
  const uint32_t bar_tempty = bar_full + kBpTempty;
  const uint32_t bar_drain = bar_full + kBpDrain;
  const uint32_t bar_sfull = bar_full + kBpSfull;
  const uint32_t bar_sempty = bar_full + kBpSempty;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBpBar + kBpWords);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kBpStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 2);  // the MMAs of both halves
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, 8);  // this half's epilogue warps of both CTAs
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_drain + 8, 1);
    for (int c = 0; c < kBpChunks; ++c) {
      mbar_init(bar_sfull + 8 * c, 1);
      mbar_init(bar_sempty + 8 * c, 8);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW32);
    tma_prefetch_desc(&tmX64);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
  tc_fence_before();
  cta_sync();
  cluster_sync_all();  // both CTAs' barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  pdl_wait();
  const int chunks = EPI == BG_EPI_DENSE ? (p.T + 255) / 256 : p.meta[META_NPB];
  const int ntiles = chunks * p.n_tiles;

  if (warp < 4) {
    setmaxnreg_dec<kBpRoleRegs>();
    if (warp == 0) {
      // ---------------- TMA producer (both CTAs) ----------------
      // completion is counted on CTA 0's full barrier, which CTA 0 arms for both CTAs' bytes
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int t = pair; t < ntiles && ok; t += npairs) {
        const BpTile d = bp_tile_at<EPI>(p, t);
        for (int kb = 0; kb < p.kb_total; ++kb) {
          if (!mbar_wait_all(bar_empty + 8 * stage, phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t sw = sbase + stage * kBpStage, fb = bar_full + 8 * stage, fb0 = mapa_shared(fb, 0);
            if (leader) mbar_arrive_expect_tx(fb, (d.tail ? 3u : 4u) * kBpHalf);
            if (G1 && d.tail) {  // 32 gate rows, the matching 32 up rows, the next 32 of each
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int wr = d.wr0 + 64 * (int)rank + 32 * j;
                tma_load_2d_pair(sw + j * (kBpHalf / 2), &tmW32, kb * 128, wr, fb0);
                tma_load_2d_pair(sw + j * (kBpHalf / 2) + kBpHalf / 4, &tmW32, kb * 128, wr + p.w_pair_off, fb0);
              }
            } else {
              tma_load_2d_pair(sw, &tmW, kb * 128, d.wr0 + (rank ? p.w_pair_off : 0), fb0);
            }
            if (d.tail)
              tma_load_2d_pair(sw + kBpHalf, &tmX64, kb * 128, d.xrow + 64 * (int)rank, fb0);
            else
              tma_load_2d_pair(sw + kBpHalf, &tmX, kb * 128, d.xrow + 128 * (int)rank, fb0);
          }
          __syncwarp();
          ++issued;
          if (++stage == kBpStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (lane == 0) {
        pdl_launch_dependents();
        if (!ok && leader) {  // let the copies already in flight land before the CTA exits
          const uint32_t first = issued > (uint32_t)kBpStages ? issued - kBpStages : 0u;
          for (uint32_t i = first; i < issued; ++i)
            mbar_wait_drain(bar_full + 8 * (i % kBpStages), (i / kBpStages) & 1u, 100000000ull);
        }
      }
      __syncwarp();
    } else if (warp < 3) {
      // ---------------- MMA issuers (CTA 0): one thread for each half of a K block ----------------
      // The thread's own instructions are the limit here: a satisfied wait takes about 70 cycles, the
      // issue 90, and one thread doing both halves with its waits in turn took longer than the MMAs
      // (600 to 1100 cycles a block for 545).  So each half has its thread, on different SM quarters,
      // and both waits of a block are polled together.
      if (leader && elect_one()) {
        const uint32_t h = warp - 1;
        const uint64_t a0 = sdesc_k_sw128(sbase + kBpHalf), b0 = sdesc_k_sw128(sbase + h * (kBpHalf / 2));
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true, any = false;
        for (int t = pair; t < ntiles && ok; t += npairs) {
          const uint32_t idesc = idesc_make(bp_tile_at<EPI>(p, t).tail ? 128 : 256, 128, true);
          for (int kb = 0; kb < p.kb_total; ++kb) {
            const uint32_t fb = bar_full + 8 * stage, eb = bar_tempty + 8 * (2 * buf + h);
            const bool full = mbar_try_wait(fb, phase), free_buf = mbar_try_wait(eb, buf_phase ^ 1u);
            if (!(full && free_buf)) {
              ok = mbar_wait_one(fb, phase, abort_flag, p.status) &&
                   mbar_wait_one(eb, buf_phase ^ 1u, abort_flag, p.status);
              if (!ok) break;
            }
            tc_fence_after();
            const uint64_t so = (uint64_t)(stage * (kBpStage >> 4));
            tc_mma_pair_kblock(tmem_base + 256u * buf + 128u * h, a0 + so, b0 + so, idesc);
            tc_commit_both(bar_tfull + 8 * (2 * buf + h));
            tc_commit_both(bar_empty + 8 * stage);
            any = true;
            if (++stage == kBpStages) {
              stage = 0;
              phase ^= 1u;
            }
            buf ^= 1;
            if (buf == 0) buf_phase ^= 1u;
          }
        }
        if (!ok && any) {  // the tensor cores must be idle before tensor memory is freed
          tc_commit_pair(bar_drain + 8 * h);
          mbar_wait_drain(bar_drain + 8 * h, 0, 100000000ull);
        }
      }
      __syncwarp();
    } else {
      // ---------------- scales (warp 3): products of row and weight scales, in chunks of K blocks ----------------
      // (the fold's threads would wait for these loads: a row's scales lie kb_total floats from the
      // next row's, so a warp's load touches 32 lines)
      float2* ring = reinterpret_cast<float2*>(smem + kBpScale);
      int chunk = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; t < ntiles && ok; t += npairs) {
        const BpTile d = bp_tile_at<EPI>(p, t);
        for (int kc = 0; kc < p.kb_total; kc += kBpChunk) {
          if (!mbar_wait_all(bar_sempty + 8 * chunk, phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          // 64 rows at a time: this warp shares its register budget with the other roles
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            const int r0 = bp_row<EPI>(d, rank, lane + 64 * hf), r1 = bp_row<EPI>(d, rank, lane + 64 * hf + 32);
            const float* x0 = p.a_scale + (size_t)(EPI != BG_EPI_DENSE || r0 < p.T ? r0 : 0) * p.kb_total;
            const float* x1 = p.a_scale + (size_t)(EPI != BG_EPI_DENSE || r1 < p.T ? r1 : 0) * p.kb_total;
            const float *wa, *wb;
            bp_scale_rows<EPI>(p, d, 64 * hf, wa, wb);
            float v0[kBpChunk], v1[kBpChunk], a[kBpChunk], b[kBpChunk];
#pragma unroll
            for (int i = 0; i < kBpChunk; ++i) {
              const int kb = min(kc + i, p.kb_total - 1);
              v0[i] = x0[kb];
              v1[i] = x1[kb];
              a[i] = wa[kb];
              b[i] = wb[kb];
            }
            float2* dst = ring + chunk * (kBpChunk * 128) + 64 * hf + lane;
#pragma unroll
            for (int i = 0; i < kBpChunk; ++i) {
              dst[i * 128] = make_float2(v0[i] * a[i], v0[i] * b[i]);
              dst[i * 128 + 32] = make_float2(v1[i] * a[i], v1[i] * b[i]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_sfull + 8 * chunk);
          if (++chunk == kBpChunks) {
            chunk = 0;
            phase ^= 1u;
          }
        }
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kBpEpiRegs>();
    // ---------------- epilogue (warps 4..11 of both CTAs) ----------------
    BpFold f;
    {
      const uint32_t q = warp & 3, h = (warp - 4) >> 2;  // tensor-memory quadrant; half of the K block
      f.bars = bar_full;
      f.tmem = tmem_base + ((q * 32) << 16) + 128u * h;
      f.tfull = bar_tfull + 8 * h;
      f.tempty = mapa_shared(bar_tempty, 0) + 8 * h;
      f.scale = sbase + kBpScale + (q * 32 + lane) * 8u;
      f.blocks = f.chunks = 0;
      f.ok = true;
    }
    int par = 0;
    for (int t = pair; t < ntiles; t += npairs) {
      // This thread's row and its two runs of `wide` sums, tensor-memory columns [0, wide) and
      // [wide, 2 wide) of its half: of box 0 and box 1, or (tail) of box hf alone.
      float2 acca[32], accb[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acca[i] = accb[i] = make_float2(0.0f, 0.0f);
      if (!bp_tile_at<EPI>(p, t).tail)
        bp_fold_tile<false>(f, p.kb_total, p.status, acca, accb);
      else
        bp_fold_tile<true>(f, p.kb_total, p.status, acca, accb);
      // the tile's place and the thread's, computed here again rather than kept through the fold
      int t_again = t, tid = threadIdx.x - 128;
      asm volatile("" : "+r"(t_again), "+r"(tid));
      const BpTile d = bp_tile_at<EPI>(p, t_again);
      const int lrow = tid & 127, h = tid >> 7;
      const int hf = d.tail ? lrow >> 6 : 0;
      const int row = bp_row<EPI>(d, rank, lrow);
      const int wide = d.tail ? 32 : 64;
      float* red = reinterpret_cast<float*>(smem + kBpRed);
      if constexpr (G1) {
        // SiLU(gate) * up of `wide` columns, the block's maximum over the two (tail: four) threads
        // of the row, then this thread's codes
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (i < wide / 2) {
            acca[i].x = silu_mul_fast(acca[i].x, accb[i].x);
            acca[i].y = silu_mul_fast(acca[i].y, accb[i].y);
            a = max_nan(a, max_nan(fabsf(acca[i].x), fabsf(acca[i].y)));
          }
        }
        float* rd = red + 256 * par;
        rd[128 * h + lrow] = a;
        named_bar_sync(1, 256);
        a = max_nan(rd[lrow], rd[128 + lrow]);
        if (d.tail) a = max_nan(a, max_nan(rd[lrow ^ 64], rd[128 + (lrow ^ 64)]));
        par ^= 1;  // (the other half of red: a slower warp may still read this one)
        const float s = block_scale_from_amax(a);
        const float r = 1.0f / s;
        if (!d.tail && __all_sync(0xffffffffu, f.ok)) {
          // 32 rows x 64 bytes of a warp by one TMA store, as bp_store_box
          const int lane_ = tid & 31;
          const uint32_t buf = sbase + kBpOut + (uint32_t)(tid >> 5) * kBpOutWarp;
          if (lane_ == 0) bulk_wait_read();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = pack_e4m3x4(acca[8 * c + 2 * j].x * r, acca[8 * c + 2 * j].y * r, acca[8 * c + 2 * j + 1].x * r,
                                 acca[8 * c + 2 * j + 1].y * r);
            sts_v4(buf + lane_ * 64u + (uint32_t)((c ^ ((lane_ >> 1) & 3)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane_ == 0) {
            tma_store_2d(&tmO, buf, d.n * 128 + 64 * h, row - lane_);
            bulk_commit();
          }
        } else if (d.tail && f.ok) {
          uint8_t* dst = static_cast<uint8_t*>(p.out) + (size_t)row * p.n_out + (size_t)d.n * 128 + 64 * hf + 32 * h;
          uint32_t c[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            c[j] = pack_e4m3x4(acca[2 * j].x * r, acca[2 * j].y * r, acca[2 * j + 1].x * r, acca[2 * j + 1].y * r);
          st_global_v8(dst, c);
        }
        if (f.ok && h == 0 && hf == 0) p.out_scale[(size_t)row * (p.n_out / 128) + d.n] = s;
      } else if (p.out_tma) {
        // GEMM2's rows stay in expert order (the combine finds them through the inverse map) and leave as
        // bf16: the outputs of a token's experts are rounded once more before their fp32 sum, about 2^-9 of
        // each, below the 2^-4 steps of the e4m3 intermediate they come from, for half the bytes written
        // here and read by the combine (0.2 ms of a layer of 8192 tokens).
        if (__all_sync(0xffffffffu, f.ok)) {
          const uint32_t buf = sbase + kBpOut + (uint32_t)(tid >> 5) * kBpOutWarp;
          const int lane_ = tid & 31, row0 = row - lane_;
          const int n = d.n * 256 + 128 * hf + 64 * h;  // columns of box 0 (tail: of box hf)
          if (EPI == BG_EPI_G2 || p.out_bf16) {
            if (!d.tail) {
              bp_store_box<true>(p, &tmO, buf, lane_, row0, n, [&](int i) { return acca[i]; });
              bp_store_box<true>(p, &tmO, buf, lane_, row0, n + 128, [&](int i) { return accb[i]; });
            } else {
              bp_store_box<true>(p, &tmO, buf, lane_, row0, n,
                                 [&](int i) { return i < 16 ? acca[i & 15] : accb[i & 15]; });
            }
          } else {
            bp_store_box<false>(p, &tmO, buf, lane_, row0, n, [&](int i) { return acca[i]; });
            if (!d.tail) {
              bp_store_box<false>(p, &tmO, buf, lane_, row0, n + 32, [&](int i) { return acca[16 + i]; });
              bp_store_box<false>(p, &tmO, buf, lane_, row0, n + 128, [&](int i) { return accb[i]; });
              bp_store_box<false>(p, &tmO, buf, lane_, row0, n + 160, [&](int i) { return accb[16 + i]; });
            } else {
              bp_store_box<false>(p, &tmO, buf, lane_, row0, n + 32, [&](int i) { return accb[i]; });
            }
          }
        }
      } else if (EPI == BG_EPI_DENSE && f.ok && row < p.T) {
        const int n = d.n * 256 + 128 * hf + 64 * h;
        if (!d.tail) {
          bp_store<32>(p, (size_t)row, n, acca);
          bp_store<32>(p, (size_t)row, n + 128, accb);
        } else {
          bp_store<16>(p, (size_t)row, n, acca);
          bp_store<16>(p, (size_t)row, n + 32, accb);
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // no row is on its way when the CTA ends
  }

  // Both CTAs finish every role (and with it every read of the other CTA's shared memory or tensor
  // memory) before either frees tensor memory or exits.
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// Clusters of 2 on a persistent grid of as many pairs as are resident at once.
template <int EPI>
cudaError_t launch_bp(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& mw32, const CUtensorMap& mx64,
                      const CUtensorMap& mo, const BgDev& p, long tiles, cudaStream_t s) {
  static bool attr_set[64] = {};
  static int max_clusters[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kern = k_gemm_block_pair<EPI>;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kBpThreads);
  cfg.dynamicSmemBytes = kBpSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(2);
  if (max_clusters[dev] == 0) {
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = -1;
    }
    max_clusters[dev] = n;
  }
  if (max_clusters[dev] < 1) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(2 * (unsigned)std::max<long>(1, std::min<long>(tiles, max_clusters[dev])));
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, mw32, mx64, mo, p);
}

}  // namespace

cudaError_t launch_gemm_block(const BlockGemmArgs& a, cudaStream_t s) {
  CUtensorMap mw, mx;
  const uint64_t x_rows = a.epi == BG_EPI_DENSE ? (uint64_t)a.T : (uint64_t)a.cap;
  if (!make_tensor_map_2d(&mw, a.w, 1, (uint64_t)a.K, (uint64_t)a.E * a.w_rows, 128u) ||
      !make_tensor_map_2d(&mx, a.x, 1, (uint64_t)a.K, x_rows, a.pair ? 128u : 16u))
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
  p.out_bf16 = a.out_bf16 ? 1 : 0;
  p.early = a.early ? 1 : 0;
  p.out_rows = (int)x_rows;
  p.a_scale = a.a_scale;
  p.w_scale = a.w_scale;
  p.sorted = a.sorted;
  p.eids = a.eids;
  p.meta = a.meta;
  p.ids = a.ids;
  p.out = a.out;
  p.out_scale = a.out_scale;
  p.status = a.status;
  if (a.pair) {
    CUtensorMap mw32, mx64, mo = {};
    if (!make_tensor_map_2d(&mw32, a.w, 1, (uint64_t)a.K, (uint64_t)a.E * a.w_rows, 32u) ||
        !make_tensor_map_2d(&mx64, a.x, 1, (uint64_t)a.K, x_rows, 64u))
      return cudaErrorInvalidValue;
    p.pblk = a.pblk;
    if (a.epi == BG_EPI_G1) {
      if (!make_tensor_map_2d(&mo, a.out, 1, (uint64_t)a.n_out, x_rows, 32u, 64u)) return cudaErrorInvalidValue;
    } else {
      p.out_tma = (long)a.n_out * (a.out_bf16 ? 2 : 4) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
      if (!p.out_tma && a.epi == BG_EPI_G2) return cudaErrorInvalidValue;
      if (p.out_tma && !make_tensor_map_2d(&mo, a.out, 2, (uint64_t)a.n_out * (a.out_bf16 ? 1 : 2), x_rows, 32u))
        return cudaErrorInvalidValue;
    }
    if (a.epi == BG_EPI_DENSE)
      return launch_bp<BG_EPI_DENSE>(mw, mx, mw32, mx64, mo, p, ((long)a.T + 255) / 256 * p.n_tiles, s);
    const long tiles = (long)(a.cap / 128) * p.n_tiles;
    if (a.epi == BG_EPI_G1) return launch_bp<BG_EPI_G1>(mw, mx, mw32, mx64, mo, p, tiles, s);
    return launch_bp<BG_EPI_G2>(mw, mx, mw32, mx64, mo, p, tiles, s);
  }
  if (a.epi == BG_EPI_DENSE) {
    const long tiles = ((long)a.T + a.nt - 1) / a.nt * p.n_tiles;
    return launch_bg_nt<BG_EPI_DENSE>(mw, mx, p, a.nt, tiles, a.num_sms, s);
  }
  const long groups = a.cap / a.nt;  // blocks of the permutation at most
  if (a.epi == BG_EPI_G1) return launch_bg_nt<BG_EPI_G1>(mw, mx, p, a.nt, groups * p.n_tiles, a.num_sms, s);
  return launch_bg_nt<BG_EPI_G2>(mw, mx, p, a.nt, groups * p.n_tiles, a.num_sms, s);
}

}  // namespace moe
