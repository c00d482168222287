// The permutation of at most 32 (token, expert) pairs by one warp, for the kernels that need it
// whole (maps for the kernels behind) or in part (slots, tile lists).
#pragma once
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

// What lane i knows of pair i: warp match gives the pair's expert group and its rank in it (lower
// flat index first), and the group leaders -- the active experts -- find their padded offsets by
// comparing expert ids over the warp.
struct SmallGroup {
  int e;             // expert, -1 for none
  int count, pad;    // pairs of the expert, padded to the block size
  int below, off;    // active experts with smaller ids; their padded rows
  int slot;          // this pair's row in expert order
  bool leader;       // the expert's first pair
  unsigned leaders;
};

// All 32 lanes of a warp; n <= 32.  Ids out of range count as none and are reported to status
// (nullable), and so are an expert's pairs past max_count.
__device__ __forceinline__ SmallGroup align_small(const int32_t* __restrict__ ids, int n, int E, int B, int* status,
                                                  int skip_minus_one, int max_count = 32) {
  const int lane = threadIdx.x & 31;
  SmallGroup g;
  g.e = -1;
  if (lane < n) {
    g.e = ids[lane];
    if (g.e < 0 || g.e >= E) {
      if (status && !(skip_minus_one && g.e == -1)) report(status, MOE_ERR_DEVICE_INDEX);
      g.e = -1;
    }
  }
  __syncwarp();
  unsigned grp = __match_any_sync(0xffffffffu, g.e);
  if (max_count < n) {
    if (g.e >= 0 && __popc(grp & ((1u << lane) - 1u)) >= max_count) {
      if (status) report(status, MOE_ERR_DEVICE_INDEX);
      g.e = -1;
    }
    __syncwarp();
    grp = __match_any_sync(0xffffffffu, g.e);
  }
  g.count = __popc(grp);
  g.leader = g.e >= 0 && lane == __ffs(grp) - 1;
  g.leaders = __ballot_sync(0xffffffffu, g.leader);
  g.pad = (g.count + B - 1) / B * B;
  g.below = 0;
  g.off = 0;
  for (int j = 0; j < n; ++j) {
    const int ej = __shfl_sync(0xffffffffu, g.e, j);
    const int pj = __shfl_sync(0xffffffffu, g.pad, j);
    if (((g.leaders >> j) & 1u) && ej < g.e) {
      ++g.below;
      g.off += pj;
    }
  }
  g.slot = g.off + __popc(grp & ((1u << lane) - 1u));
  return g;
}

// The maps of the permutation (outputs as k_align's), by the warp that holds g.
__device__ __forceinline__ void align_small_maps(const SmallGroup& g, int n, int E, int B, int32_t* __restrict__ sorted,
                                                 int32_t* __restrict__ eids, int32_t* __restrict__ npp_out,
                                                 int32_t* __restrict__ counts_out, int32_t* __restrict__ meta,
                                                 int32_t* __restrict__ inv) {
  __shared__ int s_e[32], s_off[32], s_c[32];  // active experts in ascending order
  const int lane = threadIdx.x & 31;
  int total = g.leader ? g.pad : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int nact = __popc(g.leaders);
  if (g.leader) {
    s_e[g.below] = g.e;
    s_off[g.below] = g.off;
    s_c[g.below] = g.count;
    if (meta) meta[meta_active(E) + g.below] = g.e;
  }
  if (g.e >= 0) {
    sorted[g.slot] = lane;
    if (inv) inv[lane] = g.slot;
  } else if (inv && lane < n) {
    inv[lane] = -1;
  }
  // block -> expert map and sentinel rows: each active expert's leader writes its own run
  if (g.leader) {
    for (int b = g.off / B; b < (g.off + g.pad) / B; ++b) eids[b] = g.e;
    for (int q = g.off + g.count; q < g.off + g.pad; ++q) sorted[q] = n;
  }
  __syncwarp();
  // every expert's offset and count: those of the first active expert at or above it
  // (lane x visits x, x + 32, ...: the active index lo only moves forward)
  int lo = 0;
  for (int x = lane; x < E; x += 32) {
    while (lo < nact && s_e[lo] < x) ++lo;
    const int cnt = (lo < nact && s_e[lo] == x) ? s_c[lo] : 0;
    if (meta) {
      meta[meta_offsets(E) + x] = lo < nact ? s_off[lo] : total;
      meta[meta_counts(E) + x] = cnt;
    }
    if (counts_out) counts_out[x] = cnt;
  }
  if (lane == 0) {
    *npp_out = total;
    if (meta) {
      meta[META_NPP] = total;
      meta[META_NBLK] = total / B;
      meta[META_NACT] = nact;
      meta[meta_offsets(E) + E] = total;
    }
  }
}

}  // namespace moe
