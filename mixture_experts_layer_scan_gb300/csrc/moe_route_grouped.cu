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
// redux.max, one ballot and the winning lane's rescan of its own keys.  The scores of the chosen
// experts are computed again from their logits instead of being carried next to the keys (half the
// registers; the same function of the same input, so the same bits).
#include "moe_internal.h"
#include "moe_device.cuh"

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
  int lpg;       // lanes per group
  int per_lane;  // experts per lane
  int sigmoid, group_sum, renorm;
  int by_logit;  // rank the logits themselves (softmax without bias orders like its logits)
  float scale;
};

// Order-preserving integer key of a score; NaN counts as -inf, and 0 is below every key.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0x007fffffu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kTakenKey = 0u;

__device__ __forceinline__ float sigmoid_score(float l) { return 1.0f / (1.0f + expf(-l)); }
__device__ __forceinline__ float no_nan(float v) { return v == v ? v : -INFINITY; }

template <int V>
__global__ void __launch_bounds__(kRouteWarps * 32) k_topk_grouped(const GroupedDev p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const float* __restrict__ l = p.logits + (size_t)t * p.E;
  const int group = lane / p.lpg;
  const int in_group = (lane - group * p.lpg) * p.per_lane;  // first expert of this lane inside its group
  const int first = group * p.group_size + in_group;
  const int mine = group < p.n_group ? max(0, min(p.per_lane, p.group_size - in_group)) : 0;

  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = j < mine ? l[first + j] : -INFINITY;

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
      if (j < mine) sum += expf(v[j] - m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  }
  uint32_t key[V];
  float top1 = -INFINITY, top2 = -INFINITY;  // of this lane's r
#pragma unroll
  for (int j = 0; j < V; ++j) {
    key[j] = kTakenKey;
    if (j < mine) {
      float r = v[j];
      if (!p.by_logit) {
        r = p.sigmoid ? sigmoid_score(v[j]) : expf(v[j] - m) / sum;
        if (p.bias) r += p.bias[first + j];
      }
      r = no_nan(r + 0.0f);  // (-0 ranks as +0)
      key[j] = order_key(r);
      top2 = fmaxf(top2, fminf(top1, r));
      top1 = fmaxf(top1, r);
    }
  }

  if (p.topk_group < p.n_group) {
    for (int off = 1; off < p.lpg; off <<= 1) {  // (lpg is a power of two: the butterfly stays in the group)
      const float o1 = __shfl_xor_sync(kAll, top1, off), o2 = __shfl_xor_sync(kAll, top2, off);
      top2 = fmaxf(fminf(top1, o1), fmaxf(top2, o2));
      top1 = fmaxf(top1, o1);
    }
    const float gs = (p.group_sum == 2 && p.group_size > 1) ? no_nan(top1 + top2) : top1;
    uint32_t gk = group < p.n_group ? order_key(gs + 0.0f) : kTakenKey;
    bool keep = false;
    for (int r = 0; r < p.topk_group; ++r) {
      const uint32_t best = __reduce_max_sync(kAll, gk);
      const int winner = (__ffs(__ballot_sync(kAll, gk == best)) - 1) / p.lpg;
      if (group == winner) {
        keep = true;
        gk = kTakenKey;
      }
    }
    if (!keep) {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = kTakenKey;
    }
  }

  // the k largest keys, ties to the lower expert
  uint32_t lmax = kTakenKey;
  int lj = 0;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (key[j] > lmax) {
      lmax = key[j];
      lj = j;
    }
  int my_id = 0;
  for (int r = 0; r < p.k; ++r) {
    const uint32_t best = __reduce_max_sync(kAll, lmax);
    const int winner = __ffs(__ballot_sync(kAll, lmax == best)) - 1;
    const int id = __shfl_sync(kAll, first + lj, winner);
    if (lane == r) my_id = id;
    if (lane == winner) {
      const int out = lj;
      lmax = kTakenKey;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j == out) key[j] = kTakenKey;
        if (key[j] > lmax) {
          lmax = key[j];
          lj = j;
        }
      }
    }
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
  p.lpg = 1;
  while (2 * p.lpg * p.n_group <= 32) p.lpg *= 2;
  p.per_lane = (p.group_size + p.lpg - 1) / p.lpg;
  p.sigmoid = rule.score == MOE_SCORE_SIGMOID;
  p.group_sum = rule.group_sum;
  p.renorm = rule.renorm != 0;
  p.by_logit = rule.score == MOE_SCORE_SOFTMAX && !bias && (rule.topk_group == rule.n_group || rule.group_sum == 1);
  p.scale = rule.scale;
  const dim3 grid((T + kRouteWarps - 1) / kRouteWarps), block(kRouteWarps * 32);
  if (p.per_lane <= 4) MOE_LAUNCH(k_topk_grouped<4>, grid, block, 0, s, p);
  else if (p.per_lane <= 8) MOE_LAUNCH(k_topk_grouped<8>, grid, block, 0, s, p);
  else if (p.per_lane <= 16) MOE_LAUNCH(k_topk_grouped<16>, grid, block, 0, s, p);
  else if (p.per_lane <= 32) MOE_LAUNCH(k_topk_grouped<32>, grid, block, 0, s, p);
  else MOE_LAUNCH(k_topk_grouped<64>, grid, block, 0, s, p);  // (n_group > 16: up to 1024 / 17 experts in a lane)
  return cudaGetLastError();
}

}  // namespace moe
