// Norms before and after a block: the forward kernel (moe_norm.cuh has the formulas and the rows).
#include "moe_norm.cuh"

namespace moe {

namespace {

// The sums' shared memory alternates from row to row: what a row wrote is overwritten two barriers later.
template <typename T, int W, int NV, int KIND, bool RING, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) k_norm(const __grid_constant__ NormDev p) {
  pdl_enter();
  using R = Rows<T, W, NV, RING>;
  constexpr int E2 = R::E / 2;
  constexpr bool POST = KIND != N_PRE, HOLD = THREADS <= 512;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sums[2][2][kMaxWarps];
  for (int i = threadIdx.x; i < 4 * kMaxWarps; i += blockDim.x) (&sums[0][0][0])[i] = 0.f;
  R rows(p, smem);
  __syncthreads();
  rows.start();
  if constexpr (POST) rows.fetch_token(blockIdx.x);
  float2 cw[POST ? E2 : 1], nw[E2];
  if constexpr (HOLD) {
    if constexpr (POST) rows.factor(cw);
    if (p.next_w) rows.weight(p.next_w, p.w_f32, 0, nw);
  }
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    rows.open(t);
    float (&s2)[2][kMaxWarps] = sums[rows.k & 1];
    float2 o[E2];
    rows.load(S_X, o);
    if constexpr (POST) {
      // out = res_scale x + (scale r_y G) (y post_w gate): what does not need r_y comes before its sum is there
      float2 y[E2], a = both(0.f);
      rows.load(S_Y, y);
      if constexpr (!HOLD) rows.factor(cw);
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        a = fma2(y[e], y[e], a);
        y[e] = mul2(y[e], cw[e]);
        o[e] = mul2(o[e], both(p.res_scale));
      }
      if constexpr (KIND == N_FULL) {
        float2 g[E2];
        rows.full_gate(g);
#pragma unroll
        for (int e = 0; e < E2; ++e) y[e] = mul2(y[e], g[e]);
      }
      float s = p.scale * rows.token_gate(t);
      if (p.post_w) {
        s *= rsqrtf(block_sum(a, s2[0]) * p.inv_h + p.eps);
        rows.refill(t);
      }
#pragma unroll
      for (int e = 0; e < E2; ++e) o[e] = fma2(both(s), y[e], o[e]);
      rows.store(p.out, o);
    }
    if (!POST || p.next_w) {
      float2 a = both(0.f);
      if constexpr (!HOLD) rows.weight(p.next_w, p.w_f32, 0, nw);
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        a = fma2(o[e], o[e], a);
        o[e] = mul2(o[e], nw[e]);
      }
      const float2 r = both(rsqrtf(block_sum(a, s2[1]) * p.inv_h + p.eps));
      rows.refill(t);
#pragma unroll
      for (int e = 0; e < E2; ++e) o[e] = mul2(o[e], r);
      rows.store(p.h, o);
    }
    rows.close(t);
  }
  rows.drain();
}

// (the ring's kernel, or the one without where rows do not fit or are few; the ring's registers decide for both)
template <typename T, int W, int NV, int KIND, bool RING, int THREADS>
cudaError_t launch_one(NormDev p, cudaStream_t s) {
  static int known[64] = {};
  auto kernel = k_norm<T, W, NV, KIND, RING, THREADS>;
  const int regs = norm_regs(kernel, known);
  if (!regs) return cudaErrorInvalidValue;
  const NormShape q = norm_shape<T, W>(p, regs, NV * (W / (int)sizeof(T)), p.T, RING);
  if constexpr (RING)
    if (!p.stages) return launch_one<T, W, NV, KIND, false, THREADS>(p, s);
  MOE_LAUNCH(kernel, dim3(q.grid), dim3(q.threads), q.smem, s, p);
  return cudaGetLastError();
}

template <typename T, int W, int KIND>
cudaError_t launch_kind(const NormDev& p, cudaStream_t s) {
  constexpr int N = W / sizeof(T);
  if constexpr (W == 16)
    if (p.T <= 304 && p.H <= 512 * 8) return launch_one<T, W, 8 / N, KIND, false, 512>(p, s);
  return p.H > 512 * kElems ? launch_one<T, W, kElems / N, KIND, false, 1024>(p, s)
                            : launch_one<T, W, kElems / N, KIND, true, 512>(p, s);
}
template <typename T, int W>
cudaError_t launch_width(const NormDev& p, int kind, cudaStream_t s) {
  return kind == N_PRE ? launch_kind<T, W, N_PRE>(p, s)
         : kind == N_POST ? launch_kind<T, W, N_POST>(p, s)
                          : launch_kind<T, W, N_FULL>(p, s);
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
  const bool vec = (long)a.H * (a.bf16 ? 2 : 4) % 16 == 0;
  if (a.bf16) return vec ? launch_width<__nv_bfloat16, 16>(p, kind, s) : launch_width<__nv_bfloat16, 2>(p, kind, s);
  return vec ? launch_width<float, 16>(p, kind, s) : launch_width<float, 4>(p, kind, s);
}

}  // namespace moe
