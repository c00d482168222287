// Norms before and after a block: the forward kernel (moe_norm.cuh has the formulas and the rows).
#include "moe_norm.cuh"

namespace moe {

namespace {

// The sums' shared memory alternates from row to row: what a row wrote is overwritten behind the next row's barrier.
// FAST: whole units in every thread, and both norms: nothing is asked for each unit.
// 16384 x 4096 bf16: postnorm 88.6 us (6.1 TB/s, 89 % of a copy's rate), prenorm 46.6; one row 1.7 us.
template <typename T, int NV, int KIND, bool RING, int THREADS, bool FAST, bool ODD>
__global__ void __launch_bounds__(THREADS, 1) k_norm(const __grid_constant__ NormDev p) {
  pdl_enter();
  using R = Rows<T, NV, RING, FAST, ODD>;
  constexpr int C2 = R::C2, CH = NV;
  constexpr bool POST = KIND != N_PRE, HOLD = THREADS <= 512;
  const bool post = FAST || p.post_w, next = !POST || FAST || p.next_w;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sums[2][2][THREADS / 4];
  R rows(p, smem);
  __syncthreads();
  rows.start();
  if constexpr (KIND == N_POST) rows.fetch_token(blockIdx.x);
  float2 cw[HOLD && POST ? CH : 1][C2], nw[HOLD ? CH : 1][C2];
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (POST) rows.template factor<KIND == N_POST>(c, cw[c]);
      if (next) rows.weight(p.next_w, p.w_f32, 0, c, nw[c]);
    }
  }
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    rows.open(t);
    float (&s2)[2][THREADS / 4] = sums[rows.k & 1];
    float2 o[CH][C2], y[POST ? CH : 1][C2];
    float2 a0 = both(0.f), a1 = a0, a2 = a0, a3 = a0;  // x^2, y^2, x c, c^2
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      rows.load(S_X, c, o[c]);
      if constexpr (POST) {
        if constexpr (!HOLD) rows.template factor<KIND == N_POST>(c, cw[0]);
        float2 g[C2];
        rows.load(S_Y, c, y[c]);
        if constexpr (KIND == N_FULL) rows.full_gate(c, g);
#pragma unroll
        for (int e = 0; e < C2; ++e) {
          a1 = fma2(y[c][e], y[c][e], a1);
          y[c][e] = mul2(y[c][e], cw[HOLD ? c : 0][e]);
          if constexpr (KIND == N_FULL) y[c][e] = mul2(y[c][e], rows.gate_of(g[e]));
          a2 = fma2(o[c][e], y[c][e], a2);
          a3 = fma2(y[c][e], y[c][e], a3);
        }
      }
#pragma unroll
      for (int e = 0; e < C2; ++e) a0 = fma2(o[c][e], o[c][e], a0);
    }
    float r = 0.f, b = 0.f;
    if constexpr (POST) {
      float v[4] = {flat(a0), flat(a1), flat(a2), flat(a3)};
      block_sums(v, s2[0]);
      rows.refill(t);
      b = p.scale;
      if constexpr (KIND == N_POST) b *= rows.token_gate(t).x;
      if (post) b *= rsqrtf(v[1] * p.inv_h + p.eps);
      const float pp = p.res_scale * p.res_scale * v[0], qq = b * b * v[3], ee = pp + qq + 2.f * p.res_scale * b * v[2];
      r = ee;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int e = 0; e < C2; ++e) o[c][e] = fma2(both(b), y[c][e], mul2(both(p.res_scale), o[c][e]));
        rows.store(p.out, c, o[c]);
      }
      if (next && parts_fail(pp, qq, ee, b, v[3])) {
        a0 = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < C2; ++e) a0 = fma2(o[c][e], o[c][e], a0);
        float u[1] = {flat(a0)};
        block_sums(u, s2[1]);
        r = u[0];
      }
    } else {
      float v[1] = {flat(a0)};
      block_sums(v, s2[0]);
      rows.refill(t);
      r = v[0];
    }
    if (next) {
      r = rsqrtf(r * p.inv_h + p.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if constexpr (!HOLD) rows.weight(p.next_w, p.w_f32, 0, c, nw[0]);
#pragma unroll
        for (int e = 0; e < C2; ++e) o[c][e] = mul2(mul2(o[c][e], both(r)), nw[HOLD ? c : 0][e]);
        rows.store(p.h, c, o[c]);
      }
    }
    rows.close();
  }
  rows.drain();
}

// (the ring's kernel, or the one without where rows do not fit or are few; the ring's registers decide for both)
template <typename T, int NV, int KIND, bool RING, int THREADS, bool ODD, bool FAST = false>
cudaError_t launch_one(NormDev p, cudaStream_t s) {
  if constexpr (RING && !FAST && !ODD)
    if (p.H % (32 * kElems) == 0 && (KIND == N_PRE || (p.post_w && p.next_w)))
      return launch_one<T, NV, KIND, RING, THREADS, ODD, true>(p, s);
  static int known[64] = {};
  auto kernel = k_norm<T, NV, KIND, RING, THREADS, FAST, ODD>;
  const int regs = norm_regs(kernel, known);
  if (!regs) return cudaErrorInvalidValue;
  const NormShape q = norm_shape<T>(p, regs, NV * (16 / (int)sizeof(T)), p.T, RING);
  if constexpr (RING)
    if (!p.stages) return launch_one<T, NV, KIND, false, THREADS, ODD>(p, s);
  MOE_LAUNCH(kernel, dim3(q.grid), dim3(q.threads), q.smem, s, p);
  return cudaGetLastError();
}

template <typename T, int KIND, bool ODD>
cudaError_t launch_kind(const NormDev& p, cudaStream_t s) {
  constexpr int N = 16 / sizeof(T);
  const int elems = norm_elems(p.H, N);
  if constexpr (!ODD)
    if (p.T <= 304 && elems <= 512 * 8) return launch_one<T, 8 / N, KIND, false, 512, ODD>(p, s);
  return elems > 512 * kElems ? launch_one<T, long_elems(ODD) / N, KIND, false, long_threads(ODD), ODD>(p, s)
                              : launch_one<T, kElems / N, KIND, true, 512, ODD>(p, s);
}
template <typename T, bool ODD>
cudaError_t launch_width(const NormDev& p, int kind, cudaStream_t s) {
  return kind == N_PRE ? launch_kind<T, N_PRE, ODD>(p, s)
         : kind == N_POST ? launch_kind<T, N_POST, ODD>(p, s)
                          : launch_kind<T, N_FULL, ODD>(p, s);
}

}  // namespace

NormDev norm_dev(const NormArgs& a) {
  NormDev p = {};
  p.stream[S_X] = a.x;
  p.stream[S_Y] = a.y;
  p.stream[S_DOUT] = a.d_out;
  p.stream[S_DH] = a.d_h;
  p.post_w = a.post_w;
  p.gate = a.gate;
  if (a.rule.gate == MOE_GATE_FULL) {
    p.stream[S_GATE] = a.gate;
    p.gate_ring = (a.rule.gate_dtype == MOE_BF16) == a.bf16;
  }
  p.next_w = a.next_w;
  p.out = a.out;
  p.h = a.h;
  p.d_x = a.d_x;
  p.d_y = a.d_y;
  p.d_gate = a.d_gate;
  p.T = a.T;
  p.H = a.H;
  p.inv_h = 1.0f / (float)a.H;
  p.eps = a.rule.eps;
  p.scale = a.rule.scale;
  p.res_scale = a.rule.res_scale;
  p.gate_kind = a.rule.gate;
  p.sigmoid = a.rule.gate_sigmoid != 0 && a.rule.gate != MOE_GATE_NONE;
  p.w_f32 = a.rule.w_dtype == MOE_F32;
  p.gate_f32 = a.rule.gate_dtype == MOE_F32;
  p.status = a.status;
  return p;
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  const NormDev p = norm_dev(a);
  const int kind = !a.y ? N_PRE : a.rule.gate == MOE_GATE_FULL ? N_FULL : N_POST;
  const bool odd = (long)a.H * (a.bf16 ? 2 : 4) % 16 != 0;
  if (a.bf16) return odd ? launch_width<__nv_bfloat16, true>(p, kind, s) : launch_width<__nv_bfloat16, false>(p, kind, s);
  return odd ? launch_width<float, true>(p, kind, s) : launch_width<float, false>(p, kind, s);
}

}  // namespace moe
