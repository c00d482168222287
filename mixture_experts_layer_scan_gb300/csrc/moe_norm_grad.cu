// Norms before and after a block: their gradients (moe_norm.cuh has the formulas and the rows).
#include "moe_norm.cuh"

namespace moe {

namespace {

// With u = scale D (n post_w gate) = z n cw, z = scale D and cw the columns' factor (a token's or a full gate apart):
//   d_post_w = sum_t z G n,  d_gate = sum z n post_w:  for a gate by channels both are sum_t z n times the other
//   factor, and one sum is kept;  the sum over a row of z cw n is a token gate's gradient and, times G, what d_y needs.
template <typename T, int W, int NV, int KIND, bool RING, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) k_norm_grad(const __grid_constant__ NormDev p) {
  pdl_enter();
  using R = Rows<T, W, NV, RING>;
  constexpr int N = R::N, E2 = R::E / 2;
  constexpr bool POST = KIND != N_PRE, FULL = KIND == N_FULL, HOLD = THREADS <= 512;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sums[2][3][2 * kMaxWarps];
  for (int i = threadIdx.x; i < 12 * kMaxWarps; i += blockDim.x) (&sums[0][0][0])[i] = 0.f;
  R rows(p, smem);
  __syncthreads();
  rows.start();
  if constexpr (POST) rows.fetch_token(blockIdx.x);
  const bool dh = p.stream[S_DH] != nullptr, dout = p.stream[S_DOUT] != nullptr;
  float2 cw[POST ? E2 : 1], nw[E2], acc_n[E2], acc_s[POST ? E2 : 1];
#pragma unroll
  for (int e = 0; e < E2; ++e) {
    acc_n[e] = nw[e] = both(0.f);
    if constexpr (POST) acc_s[e] = both(0.f);
  }
  if constexpr (HOLD) {
    if constexpr (POST) rows.factor(cw);
    if (dh) rows.weight(p.next_w, p.w_f32, 0, nw);
  }
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    rows.open(t);
    float (&s3)[3][2 * kMaxWarps] = sums[rows.k & 1];
    float ry = 1.0f, tok = 1.0f;
    if constexpr (POST) {
      if (p.post_w) {
        float2 y[E2], a = both(0.f);
        rows.load(S_Y, y);
#pragma unroll
        for (int e = 0; e < E2; ++e) a = fma2(y[e], y[e], a);
        ry = rsqrtf(block_sum(a, s3[0]) * p.inv_h + p.eps);
        rows.refill(t);
      }
      tok = rows.token_gate(t);
      if constexpr (!HOLD) rows.factor(cw);
    }
    if constexpr (!HOLD)
      if (dh) rows.weight(p.next_w, p.w_f32, 0, nw);
    const float sy = p.scale * tok * ry;
    float r = 0.f, m = 0.f;  // 1 / rms of out, mean(g n) of the next norm
    auto forward = [&](float2 (&o)[E2], float2 (&y)[POST ? E2 : 1], float2 (&g)[FULL ? E2 : 1]) {
      rows.load(S_X, o);
      if constexpr (POST) {
        rows.load(S_Y, y);
        if constexpr (FULL) rows.full_gate(g);
#pragma unroll
        for (int e = 0; e < E2; ++e) {
          float2 b = mul2(y[e], cw[e]);
          if constexpr (FULL) b = mul2(b, g[e]);
          o[e] = fma2(both(sy), b, mul2(both(p.res_scale), o[e]));
        }
      }
    };
    if (dh) {
      float2 o[E2], y[POST ? E2 : 1], g[FULL ? E2 : 1], d[E2], a = both(0.f), b = both(0.f);
      forward(o, y, g);
      rows.load(S_DH, d);
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        a = fma2(o[e], o[e], a);
        b = fma2(o[e], mul2(d[e], nw[e]), b);
      }
      const float2 s = block_sum2(a, b, s3[1]);
      rows.refill(t);
      r = rsqrtf(s.x * p.inv_h + p.eps);
      m = s.y * r * p.inv_h;
    }
    float2 gn[E2];  // D, then the gradient in n (but for a token's gate)
    float2 a = both(0.f);
    {
      float2 o[E2], y[POST ? E2 : 1], g[FULL ? E2 : 1], d[E2];
      forward(o, y, g);
      if (POST && dout) {
        rows.load(S_DOUT, gn);
      } else {
#pragma unroll
        for (int e = 0; e < E2; ++e) gn[e] = both(0.f);
      }
      if (dh) {
        rows.load(S_DH, d);
#pragma unroll
        for (int e = 0; e < E2; ++e) {
          const float2 nn = mul2(o[e], both(r));
          acc_n[e] = fma2(d[e], nn, acc_n[e]);
          gn[e] = fma2(both(r), fma2(nn, both(-m), mul2(d[e], nw[e])), gn[e]);
        }
      }
      if constexpr (!POST) {
        rows.store(p.d_x, gn);
      } else {
#pragma unroll
        for (int e = 0; e < E2; ++e) o[e] = mul2(gn[e], both(p.res_scale));
        rows.store(p.d_x, o);
#pragma unroll
        for (int e = 0; e < E2; ++e) {
          const float2 z = mul2(gn[e], both(p.scale)), n = mul2(y[e], both(ry));
          const float2 zc = mul2(z, cw[e]), u = mul2(zc, n);
          if constexpr (FULL) {
            gn[e] = mul2(zc, g[e]);
            acc_s[e] = fma2(mul2(z, g[e]), n, acc_s[e]);
            a = fma2(u, g[e], a);
            // d_gate, in place of out
            o[e] = p.sigmoid ? mul2(u, make_float2(g[e].x * (1.0f - g[e].x), g[e].y * (1.0f - g[e].y))) : u;
          } else {
            gn[e] = zc;
            acc_s[e] = fma2(mul2(z, both(tok)), n, acc_s[e]);
            a = add2(u, a);
          }
        }
        if constexpr (FULL) {
          if (p.d_gate) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              if (!rows.has(i)) break;
              float f[N];
#pragma unroll
              for (int c = 0; c < N; ++c) f[c] = R::pick(o, i * N + c);
              const size_t to = rows.at + (size_t)rows.vec(i) * N;
              if (p.gate_f32) {
#pragma unroll
                for (int c = 0; c < N; ++c) static_cast<float*>(p.d_gate)[to + c] = f[c];
              } else {
                using G = typename Word<N * 2>::type;
                *reinterpret_cast<G*>(static_cast<uint16_t*>(p.d_gate) + to) = narrow<__nv_bfloat16, N * 2>(f);
              }
            }
          }
        }
      }
    }
    if constexpr (POST) {
      float mean = 0.f;
      if (p.post_w || p.gate_kind == MOE_GATE_TOKEN) {
        const float s = block_sum(a, s3[2]);
        rows.refill(t);
        mean = s * p.inv_h;
        if (p.gate_kind == MOE_GATE_TOKEN && p.d_gate && threadIdx.x == 0)
          static_cast<float*>(p.d_gate)[t] = p.sigmoid ? s * tok * (1.0f - tok) : s;
      }
      if (p.post_w) {
        float2 y[E2];
        rows.load(S_Y, y);
        const float2 c0 = both(tok * ry), c1 = both(-mean * ry);
#pragma unroll
        for (int e = 0; e < E2; ++e) gn[e] = mul2(c0, fma2(c1, y[e], gn[e]));
      } else {
#pragma unroll
        for (int e = 0; e < E2; ++e) gn[e] = mul2(both(tok), gn[e]);
      }
      rows.store(p.d_y, gn);
    }
    rows.close(t);
  }
  rows.drain();
  // partial sums
  const size_t plane = (size_t)gridDim.x * p.H;
  float* part = p.part + (size_t)blockIdx.x * p.H;
  auto store = [&](float* to, const float2 (&f)[E2]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!rows.has(i)) break;
#pragma unroll
      for (int c = 0; c < N; ++c) to[(size_t)rows.vec(i) * N + c] = R::pick(f, i * N + c);
    }
  };
  if (p.sum_next) store(part + plane, acc_n);
  if constexpr (POST) {
    float2 f[E2], g[E2];
    if (p.sum_gate) {
      rows.channel_gate(g);
#pragma unroll
      for (int e = 0; e < E2; ++e) f[e] = both(1.f);
      if (p.post_w) rows.weight(p.post_w, p.w_f32, 0, f);
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        f[e] = mul2(f[e], acc_s[e]);
        if (p.sigmoid) f[e] = mul2(f[e], make_float2(g[e].x * (1.0f - g[e].x), g[e].y * (1.0f - g[e].y)));
      }
      store(part + 2 * plane, f);
    }
    if (p.sum_post) {
#pragma unroll
      for (int e = 0; e < E2; ++e) f[e] = acc_s[e];
      if (p.gate_kind == MOE_GATE_CHANNEL) {
        rows.channel_gate(g);
#pragma unroll
        for (int e = 0; e < E2; ++e) f[e] = mul2(f[e], g[e]);
      }
      store(part, f);
    }
  }
}

// out[z][c] = sum_g part[z][g][c], 32 columns to a CTA, its warps' runs of rows added in their order
struct SumDev {
  const float* part;
  float* out[3];
  int rows, H;
};
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) k_sum_rows(const SumDev p) {
  pdl_enter();
  __shared__ float s[kSumWarps][32];
  float* out = p.out[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* part = p.part + (size_t)blockIdx.y * p.rows * p.H + c;
  const int per = (p.rows + kSumWarps - 1) / kSumWarps, g0 = min(p.rows, warp * per), g1 = min(p.rows, g0 + per);
  float a = 0.f;
  if (c < p.H) {
#pragma unroll 16
    for (int g = g0; g < g1; ++g) a += part[(size_t)g * p.H];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < p.H) {
    a = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) a += s[w][lane];
    out[c] = a;
  }
}

template <typename T, int W, int NV, int KIND, bool RING, int THREADS>
cudaError_t launch_one(NormDev p, int most, int* grid, cudaStream_t s) {
  static int known[64] = {};
  auto kernel = k_norm_grad<T, W, NV, KIND, RING, THREADS>;
  const int regs = norm_regs(kernel, known);
  if (!regs) return cudaErrorInvalidValue;
  const NormShape q = norm_shape<T, W>(p, regs, kElems, most, RING);
  if constexpr (RING)
    if (!p.stages) return launch_one<T, W, NV, KIND, false, THREADS>(p, most, grid, s);
  *grid = q.grid;
  MOE_LAUNCH(kernel, dim3(q.grid), dim3(q.threads), q.smem, s, p);
  return cudaGetLastError();
}

template <typename T, int W, int KIND>
cudaError_t launch_kind(const NormDev& p, int most, int* grid, cudaStream_t s) {
  constexpr int NV = kElems / (W / sizeof(T));
  return p.H > 512 * kElems ? launch_one<T, W, NV, KIND, false, 1024>(p, most, grid, s)
                            : launch_one<T, W, NV, KIND, true, 512>(p, most, grid, s);
}
template <typename T, int W>
cudaError_t launch_width(const NormDev& p, int kind, int most, int* grid, cudaStream_t s) {
  return kind == N_PRE ? launch_kind<T, W, N_PRE>(p, most, grid, s)
         : kind == N_POST ? launch_kind<T, W, N_POST>(p, most, grid, s)
                          : launch_kind<T, W, N_FULL>(p, most, grid, s);
}

}  // namespace

// Rows of partial sums of a gradient: its CTAs at most (two of 256 threads to an SM).
int norm_grad_rows(int T, int H) { return std::min(T, 152 * norm_ctas(norm_threads(H, kElems), 128)); }

cudaError_t launch_norm_grad(const NormArgs& a, cudaStream_t s) {
  NormDev p = norm_dev(a);
  p.part = static_cast<float*>(a.workspace);
  p.sum_post = a.d_post_w != nullptr;
  p.sum_next = a.d_next_w != nullptr;
  p.sum_gate = a.rule.gate == MOE_GATE_CHANNEL && a.d_gate;
  const int kind = !a.y ? N_PRE : a.rule.gate == MOE_GATE_FULL ? N_FULL : N_POST;
  const bool vec = (long)a.H * (a.bf16 ? 2 : 4) % 16 == 0;
  const int most = norm_grad_rows(a.T, a.H);
  int rows = 0;
  cudaError_t e;
  if (a.bf16) e = vec ? launch_width<__nv_bfloat16, 16>(p, kind, most, &rows, s) : launch_width<__nv_bfloat16, 2>(p, kind, most, &rows, s);
  else e = vec ? launch_width<float, 16>(p, kind, most, &rows, s) : launch_width<float, 4>(p, kind, most, &rows, s);
  if (e != cudaSuccess || !(p.sum_post || p.sum_next || p.sum_gate)) return e;
  SumDev q = {};
  q.part = p.part;
  q.out[0] = a.d_post_w;
  q.out[1] = a.d_next_w;
  q.out[2] = p.sum_gate ? static_cast<float*>(a.d_gate) : nullptr;
  q.rows = rows;
  q.H = a.H;
  MOE_LAUNCH(k_sum_rows, dim3((a.H + 31) / 32, 3), dim3(32 * kSumWarps), 0, s, q);
  return cudaGetLastError();
}

}  // namespace moe
