// Routing by expert groups: sigmoid or softmax scores, a bias that steers the choice but not the
// weights, the best groups, the k best experts in them, and the weights renormalised and scaled.
//
//   s = sigmoid(l) or softmax(l);  r = s + bias
//   group score = largest r of the group, or the sum of its two largest
//   ids = the k largest r inside the topk_group best groups (ties: lower group, lower expert)
//   w   = s[ids] (/ their sum) * scale
//
// One warp per token, one pass over its logits.  Every group is owned by the same number of lanes
// (a power of two, so its top two values merge by butterfly shuffles), each lane owning consecutive
// experts, which stay in registers as integer keys that order like r.  Consecutive ownership makes
// the lowest lane of a tie the one with the lowest expert, so a round of the selection is one
// redux.max, one ballot and one shuffle.  Every lane knows its two best keys beforehand: only a lane
// chosen twice looks through its keys again (1.5 times for 8 of 256 experts, instead of at every
// round).  The scores of the chosen experts are computed again from their logits instead of being
// carried next to the keys (half the registers; the same function of the same input, so the same
// bits).  Bound by the instructions of the scores and the rounds (about 1000 a token, 71 % of the issue
// slots), not by the 4 bytes a logit: 16384 tokens, top-8 of 256, 4 of 8 groups, 16.4 us, 1.1 TB/s.
#include <type_traits>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouteWarps = 8;

struct GroupedDev {
  const float* logits;
  const float* bias;  // nullable
  float* w;
  int32_t* ids;
  int T, E, k;
  int n_group, topk_group, group_size;
  int lpg_log2;  // lanes per group: 2^lpg_log2
  int per_lane;  // experts per lane
  int sigmoid, group_sum, renorm;
  int by_logit;  // rank the logits themselves (softmax without bias orders like its logits)
  float scale;
};

// Order-preserving integer key of a score that is no NaN; 0 is below every key.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
constexpr uint32_t kTakenKey = 0u;

__device__ __forceinline__ float sigmoid_score(float l) { return __frcp_rn(1.0f + expf(-l)); }
__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }

// A lane's two best keys and their places; a later equal key does not displace an earlier one.
struct Best2 {
  uint32_t m1 = kTakenKey, m2 = kTakenKey;
  int j1 = 0, j2 = 0;
  __device__ __forceinline__ void add(uint32_t key, int j) {
    const bool first = key > m1, second = key > m2;
    m2 = first ? m1 : second ? key : m2;
    j2 = first ? j1 : second ? j : j2;
    m1 = first ? key : m1;
    j1 = first ? j : j1;
  }
};

// FULL: every lane owns exactly V experts, at 16-byte boundaries.
template <int V, bool FULL>
__global__ void __launch_bounds__(kRouteWarps * 32) k_topk_grouped(const GroupedDev p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const float* __restrict__ l = p.logits + (size_t)t * p.E;
  const int group = lane >> p.lpg_log2;
  const int in_group = (lane & ((1 << p.lpg_log2) - 1)) * p.per_lane;  // first expert of this lane inside its group
  const int first = group * p.group_size + in_group;
  const int mine = FULL ? V : group < p.n_group ? max(0, min(p.per_lane, p.group_size - in_group)) : 0;

  float v[V];
  if constexpr (FULL) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 q = *reinterpret_cast<const float4*>(l + first + j);
      v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = j < mine ? l[first + j] : -INFINITY;
  }

  // scores
  float m = 0.0f, sum = 1.0f;
  if (!p.sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, v[j]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (FULL || j < mine) sum += expf(v[j] - m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  }
  uint32_t key[V];
  if (p.by_logit) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = v[j] + 0.0f;  // (-0 ranks as +0)
  } else {
    if (p.sigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = sigmoid_score(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = expf(v[j] - m) / sum;
    }
    if (p.bias) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (FULL || j < mine) v[j] += p.bias[first + j];
    }
  }
  float top1 = -INFINITY, top2 = -INFINITY;  // of this lane's r
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float r = no_nan(v[j]);
    key[j] = (FULL || j < mine) ? order_key(r) : kTakenKey;
    if (FULL || j < mine) {
      top2 = fmaxf(top2, fminf(top1, r));
      top1 = fmaxf(top1, r);
    }
  }

  bool keep = mine > 0;
  if (p.topk_group < p.n_group) {
    for (int off = 1; off < (1 << p.lpg_log2); off <<= 1) {  // (the butterfly stays in the group)
      const float o1 = __shfl_xor_sync(kAll, top1, off), o2 = __shfl_xor_sync(kAll, top2, off);
      top2 = fmaxf(fminf(top1, o1), fmaxf(top2, o2));
      top1 = fmaxf(top1, o1);
    }
    const float gs = (p.group_sum == 2 && p.group_size > 1) ? no_nan(top1 + top2) : top1;
    uint32_t gk = group < p.n_group ? order_key(gs + 0.0f) : kTakenKey;
    keep = false;
    for (int r = 0; r < p.topk_group; ++r) {
      const uint32_t best = __reduce_max_sync(kAll, gk);
      const int winner = (__ffs(__ballot_sync(kAll, gk == best)) - 1) >> p.lpg_log2;
      if (group == winner) {
        keep = mine > 0;
        gk = kTakenKey;
      }
    }
  }

  // the k largest keys, ties to the lower expert
  Best2 b;
#pragma unroll
  for (int j = 0; j < V; ++j) b.add(key[j], j);
  if (!keep) b.m1 = b.m2 = kTakenKey;
  using Mask = std::conditional_t<V <= 32, uint32_t, unsigned long long>;
  Mask taken = 0;  // this lane's experts chosen so far
  int my_id = 0;
  bool second = false;  // m1 is already the second of a look through the keys
  for (int r = 0; r < p.k; ++r) {
    const uint32_t best = __reduce_max_sync(kAll, b.m1);
    const int winner = __ffs(__ballot_sync(kAll, b.m1 == best)) - 1;
    const int id = __shfl_sync(kAll, first + b.j1, winner);
    if (lane == r) my_id = id;
    bool look = false;
    if (lane == winner) {
      taken |= Mask(1) << b.j1;
      b.m1 = b.m2;
      b.j1 = b.j2;
      look = second;
      second = true;
    }
    if (look) {  // (one lane: the others wait for it)
      b = Best2();
#pragma unroll
      for (int j = 0; j < V; ++j) b.add((taken >> j) & 1 ? kTakenKey : key[j], j);
      second = false;
    }
    __syncwarp();
  }

  float s = 0.0f;
  if (lane < p.k) {
    const float x = l[my_id];
    s = p.sigmoid ? sigmoid_score(x) : expf(x - m) / sum;
  }
  if (p.renorm) {
    float tot = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) tot += __shfl_xor_sync(kAll, tot, off);
    s = tot == 0.0f ? 0.0f : s / tot;
  }
  if (lane < p.k) {
    p.ids[(size_t)t * p.k + lane] = my_id;
    p.w[(size_t)t * p.k + lane] = s * p.scale;
  }
}

template <int V>
cudaError_t launch_inst(const GroupedDev& p, bool full, cudaStream_t s) {
  const dim3 grid((p.T + kRouteWarps - 1) / kRouteWarps), block(kRouteWarps * 32);
  if constexpr (V <= 32) {  // (64 experts in a lane are never all of a power of two)
    if (full) {
      MOE_LAUNCH((k_topk_grouped<V, true>), grid, block, 0, s, p);
      return cudaGetLastError();
    }
  }
  MOE_LAUNCH((k_topk_grouped<V, false>), grid, block, 0, s, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_topk_grouped(const float* logits, const float* bias, int T, int E, int k,
                                const moe_route_rule& rule, float* w, int32_t* ids, cudaStream_t s) {
  GroupedDev p = {};
  p.logits = logits;
  p.bias = bias;
  p.w = w;
  p.ids = ids;
  p.T = T;
  p.E = E;
  p.k = k;
  p.n_group = rule.n_group;
  p.topk_group = rule.topk_group;
  p.group_size = E / rule.n_group;
  p.lpg_log2 = 0;
  while ((2 << p.lpg_log2) * p.n_group <= 32) ++p.lpg_log2;
  const int lpg = 1 << p.lpg_log2;
  p.per_lane = (p.group_size + lpg - 1) / lpg;
  p.sigmoid = rule.score == MOE_SCORE_SIGMOID;
  p.group_sum = rule.group_sum;
  p.renorm = rule.renorm != 0;
  p.by_logit = rule.score == MOE_SCORE_SOFTMAX && !bias && (rule.topk_group == rule.n_group || rule.group_sum == 1);
  p.scale = rule.scale;
  // every lane full, its logits at 16-byte boundaries (powers of two, mostly)
  const int v = p.per_lane <= 4 ? 4 : p.per_lane <= 8 ? 8 : p.per_lane <= 16 ? 16 : p.per_lane <= 32 ? 32 : 64;
  const bool full = p.per_lane == v && lpg * v == p.group_size && lpg * p.n_group == 32;
  switch (v) {
    case 4: return launch_inst<4>(p, full, s);
    case 8: return launch_inst<8>(p, full, s);
    case 16: return launch_inst<16>(p, full, s);
    case 32: return launch_inst<32>(p, full, s);
    default: return launch_inst<64>(p, false, s);  // (n_group > 16: up to 1024 / 17 experts in a lane)
  }
}

}  // namespace moe
