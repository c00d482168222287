// Norms before and after a block: their gradients (moe_norm.cuh has the formulas and the rows).
#include "moe_norm.cuh"

namespace moe {

namespace {

// Threads for which the prenorm's registers are held to what two CTAs have room for: with one, which takes a row at a
// time, 6000 x 5120 bf16 took 45 us, with two 34.
constexpr int kTwoCtas = 320;

// With z = scale G D (G a token's gate) and cw the columns' factor: d_post_w = sum_t z gate n and d_gate = sum_t z n post_w.
// For a gate by channels both are sum_t z n times the other factor, and one sum is kept.
// FAST: whole units in every thread, both norms and both incoming gradients: nothing is asked for each unit.
// 8192 x 4096 bf16: postnorm 72 us with the sums over CTAs (5.6 TB/s), prenorm 37; 4096 x 2047, off the 16-byte grid,
// prenorm 17.7 (4096 x 2048: 15.3).
template <typename T, int NV, int KIND, bool RING, int THREADS, bool FAST, bool ODD>
__global__ void __launch_bounds__(THREADS, THREADS == kTwoCtas ? 2 : 1) k_norm_grad(const __grid_constant__ NormDev p) {
  pdl_enter();
  using R = Rows<T, NV, RING, FAST, ODD>;
  constexpr int N = R::N, C2 = R::C2, CH = NV, CP = KIND != N_PRE ? CH : 1;
  constexpr bool POST = KIND != N_PRE, FULL = KIND == N_FULL, HOLD = THREADS <= 512;
  // A token gate's slope, behind the rows: in the loop it would hold a register (8192 x 4096 without the next norm 81.4 us, so
  // 78.7).  FAST, where the registers lie otherwise, has it there (8192 x 4096: 72 us, so 85), and so have few rows, for which
  // a way to memory and back counts (64 x 4096 6.2 us, so 6.7).
  constexpr bool BEHIND = KIND == N_POST && RING && !FAST;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sums[2][2][THREADS / 4];
  R rows(p, smem);
  __syncthreads();
  rows.start();
  if constexpr (POST && !FULL) rows.fetch_token(blockIdx.x);
  const bool dh = FAST || !POST || p.stream[S_DH], dout = FAST || p.stream[S_DOUT], post = FAST || p.post_w;
  float2 cw[HOLD ? CP : 1][C2], nw[HOLD ? CH : 1][C2], acc_n[CH][C2], acc_s[CP][C2];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < C2; ++e) {
      acc_n[c][e] = both(0.f);
      if constexpr (POST) acc_s[c][e] = both(0.f);
    }
  auto weights = [&](int c, float2 (&f)[C2], float2 (&n)[C2]) {
    if constexpr (POST) rows.template factor<!FULL>(c, f);
    if (dh) {
      rows.weight(p.next_w, p.w_f32, 0, c, n);
    } else {
#pragma unroll
      for (int e = 0; e < C2; ++e) n[e] = both(0.f);
    }
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) weights(c, cw[POST ? c : 0], nw[c]);
  }
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    rows.open(t);
    float (&s2)[2][THREADS / 4] = sums[rows.k & 1];
    // x, c = y post_w gate and e = d_h next_w of a chunk
    auto inputs = [&](int c, float2 (&x)[C2], float2 (&y)[C2], float2 (&yc)[C2], float2 (&d)[C2], float2 (&e)[C2], float2 (&g)[C2]) {
      if constexpr (!HOLD) weights(c, cw[0], nw[0]);
      rows.load(S_X, c, x);
      if constexpr (POST) {
        rows.load(S_Y, c, y);
        if constexpr (FULL) rows.full_gate(c, g);
#pragma unroll
        for (int i = 0; i < C2; ++i) {
          yc[i] = mul2(y[i], cw[HOLD ? c : 0][i]);
          if constexpr (FULL) yc[i] = mul2(yc[i], rows.gate_of(g[i]));
        }
      }
      rows.load(S_DH, c, d, dh);
#pragma unroll
      for (int i = 0; i < C2; ++i) e[i] = mul2(d[i], nw[HOLD ? c : 0][i]);
    };
    float2 xx = both(0.f), yy = xx, xc = xx, cc = xx, xe = xx, ce = xx, dc = xx;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float2 x[C2], y[C2], yc[C2], d[C2], e[C2], g[C2];
      inputs(c, x, y, yc, d, e, g);
#pragma unroll
      for (int i = 0; i < C2; ++i) {
        xx = fma2(x[i], x[i], xx);
        xe = fma2(x[i], e[i], xe);
        if constexpr (POST) {
          yy = fma2(y[i], y[i], yy);
          xc = fma2(x[i], yc[i], xc);
          cc = fma2(yc[i], yc[i], cc);
          ce = fma2(yc[i], e[i], ce);
        }
      }
      if constexpr (POST) {
        rows.load(S_DOUT, c, d, dout);
#pragma unroll
        for (int i = 0; i < C2; ++i) dc = fma2(d[i], yc[i], dc);
      }
    }
    float ry = 1.f, tok = 1.f, tok_slope = 1.f, b = 0.f, r, m, mean = 0.f;  // r: 1 / rms of out; m: mean(e out r)
    if constexpr (POST) {
      float v[7] = {flat(xx), flat(yy), flat(xc), flat(cc), flat(xe), flat(ce), flat(dc)};
      block_sums(v, s2[0]);
      rows.refill(t);
      if constexpr (!FULL) {
        const float2 tg = rows.token_gate(t);
        tok = tg.x;
        tok_slope = tg.y;
      }
      if (post) ry = rsqrtf(v[1] * p.inv_h + p.eps);
      b = p.scale * tok * ry;
      const float pp = p.res_scale * p.res_scale * v[0], qq = b * b * v[3];
      float ee = pp + qq + 2.f * p.res_scale * b * v[2], oe = p.res_scale * v[4] + b * v[5];
      // sums over the row of c d_out, c e and c out
      float sd = v[6], se = v[5], so = p.res_scale * v[2] + b * v[3];
      if (dh && parts_fail(pp, qq, ee, b, v[3])) {
        float2 a[5] = {};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float2 x[C2], y[C2], yc[C2], d[C2], e[C2], g[C2];
          inputs(c, x, y, yc, d, e, g);
          rows.load(S_DOUT, c, d, dout);
#pragma unroll
          for (int i = 0; i < C2; ++i) {
            x[i] = fma2(both(b), yc[i], mul2(both(p.res_scale), x[i]));
            yc[i] = mul2(yc[i], both(ry));  // (so that its products stay in range)
            a[0] = fma2(x[i], x[i], a[0]);
            a[1] = fma2(x[i], e[i], a[1]);
            a[2] = fma2(yc[i], d[i], a[2]);
            a[3] = fma2(yc[i], e[i], a[3]);
            a[4] = fma2(yc[i], x[i], a[4]);
          }
        }
        float u[5] = {flat(a[0]), flat(a[1]), flat(a[2]), flat(a[3]), flat(a[4])};
        block_sums(u, s2[1]);
        ee = u[0];
        oe = u[1];
        sd = u[2];
        se = u[3];
        so = u[4];
      } else {
        sd *= ry;
        se *= ry;
        so *= ry;
      }
      r = dh ? rsqrtf(ee * p.inv_h + p.eps) : 0.f;
      m = dh ? oe * r * p.inv_h : 0.f;
      // sum over the row of scale D c, which is a token gate's gradient times r_y's inverse
      const float u = p.scale * (dh ? sd + r * se - r * r * m * so : sd);
      mean = u * p.inv_h;
      if (!FULL && p.gate_kind == MOE_GATE_TOKEN && p.d_gate && threadIdx.x == 0)
        static_cast<float*>(p.d_gate)[t] = BEHIND ? u : u * tok_slope;
    } else {
      float v[2] = {flat(xx), flat(xe)};
      block_sums(v, s2[0]);
      rows.refill(t);
      r = rsqrtf(v[0] * p.inv_h + p.eps);
      m = v[1] * r * p.inv_h;
    }
    const float2 r2 = both(r), rm = both(-r * r * m), z2 = both(p.scale * tok), ry2 = both(ry);
    const float2 c1 = both(post ? -mean * tok * ry * ry : 0.f);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float2 x[C2], y[C2], yc[C2], d[C2], e[C2], g[C2], D[C2];
      inputs(c, x, y, yc, d, e, g);
      if constexpr (POST) {
        rows.load(S_DOUT, c, D, dout);
      } else {
#pragma unroll
        for (int i = 0; i < C2; ++i) D[i] = both(0.f);
      }
#pragma unroll
      for (int i = 0; i < C2; ++i) {
        if constexpr (POST) x[i] = fma2(both(b), yc[i], mul2(both(p.res_scale), x[i]));  // out
        if (dh) {  // (without h nothing depends on out, which may be infinite or NaN)
          acc_n[c][i] = fma2(d[i], mul2(x[i], r2), acc_n[c][i]);
          D[i] = fma2(r2, e[i], fma2(rm, x[i], D[i]));
        }
      }
      if constexpr (!POST) {
        rows.store(p.d_x, c, D);
      } else {
#pragma unroll
        for (int i = 0; i < C2; ++i) x[i] = mul2(D[i], both(p.res_scale));
        rows.store(p.d_x, c, x);
#pragma unroll
        for (int i = 0; i < C2; ++i) {
          float2 z = mul2(D[i], z2);
          const float2 n = mul2(y[i], ry2);
          if constexpr (FULL) {  // d_gate, in place of out
            const float2 u = mul2(mul2(z, cw[HOLD ? c : 0][i]), n);
            x[i] = p.sigmoid ? mul2(u, R::slope_of(g[i])) : u;
            z = mul2(z, rows.gate_of(g[i]));
          }
          acc_s[c][i] = fma2(z, n, acc_s[c][i]);
          z = mul2(z, cw[HOLD ? c : 0][i]);
          D[i] = mul2(ry2, z);  // d_y, which without a norm does not depend on y
          if (post) D[i] = fma2(c1, y[i], D[i]);
        }
        rows.store(p.d_y, c, D);
        if constexpr (FULL) {
          if (p.d_gate) {
            if (p.gate_f32 == (sizeof(T) == 4)) {
              rows.store(p.d_gate, c, x);
            } else if (rows.has(c)) {  // (a gate of the other type)
#pragma unroll
              for (int k = 0; k < N; ++k) {
                if (!rows.inside(c, k)) continue;
                const size_t to = rows.at + rows.column(c) + k;
                if (p.gate_f32) static_cast<float*>(p.d_gate)[to] = R::pick(x, k);
                else static_cast<__nv_bfloat16*>(p.d_gate)[to] = __float2bfloat16_rn(R::pick(x, k));
              }
            }
          }
        }
      }
    }
    rows.close();
  }
  rows.drain();
  // partial sums
  const size_t plane = (size_t)gridDim.x * norm_pitch(p.H);
  float* part = p.part + (size_t)blockIdx.x * norm_pitch(p.H);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (p.sum_next) rows.store_part(part + plane, c, acc_n[c]);
    if constexpr (POST) {
      float2 f[C2], g[C2], gs[C2];
      if (!FULL && p.gate_kind == MOE_GATE_CHANNEL) rows.channel_gate(c, g, gs);
      if (!FULL && p.sum_gate) {
#pragma unroll
        for (int i = 0; i < C2; ++i) f[i] = both(1.f);
        if (p.post_w) rows.weight(p.post_w, p.w_f32, 0, c, f);
#pragma unroll
        for (int i = 0; i < C2; ++i) f[i] = mul2(mul2(f[i], acc_s[c][i]), gs[i]);
        rows.store_part(part + 2 * plane, c, f);
      }
      if (p.sum_post) {
#pragma unroll
        for (int i = 0; i < C2; ++i) f[i] = !FULL && p.gate_kind == MOE_GATE_CHANNEL ? mul2(acc_s[c][i], g[i]) : acc_s[c][i];
        rows.store_part(part, c, f);
      }
    }
  }
  if constexpr (BEHIND)
    if (p.gate_kind == MOE_GATE_TOKEN && p.d_gate && p.sigmoid) {
      __syncthreads();
#pragma unroll 1
      for (long t = blockIdx.x + (long)threadIdx.x * gridDim.x; t < p.T; t += (long)blockDim.x * gridDim.x)
        static_cast<float*>(p.d_gate)[t] *= sigmoid<T>(load_one(p.gate, p.gate_f32, t)).y;
    }
}

// out[z][c] = sum_g part[z][g][lead(g) + c]: COLS columns to a CTA, the runs of rows of its threads added in their
// order.  lead(g) is where row g of the tensors begins in its first unit of n elements.
struct SumDev {
  const float* part[3];
  float* out[3];
  int rows, H, n;
};
template <int THREADS, int COLS, bool ODD>
__global__ void __launch_bounds__(THREADS) k_sum_rows(const SumDev p) {
  pdl_wait();
  constexpr int RUNS = THREADS / COLS;
  __shared__ float s[RUNS][COLS];
  const int col = threadIdx.x % COLS, run = threadIdx.x / COLS, c = blockIdx.x * COLS + col;
  const int per = (p.rows + RUNS - 1) / RUNS, g0 = min(p.rows, run * per), g1 = min(p.rows, g0 + per);
  float a = 0.f;
  if (c < p.H) {
    const int pitch = norm_pitch(p.H);
    const float* part = p.part[blockIdx.y] + (size_t)g0 * pitch + c;
    int lead = ODD ? g0 * p.H & (p.n - 1) : 0;
#pragma unroll 16
    for (int g = g0; g < g1; ++g) {
      a += part[lead];
      part += pitch;
      if (ODD) lead = (lead + p.H) & (p.n - 1);
    }
  }
  s[run][col] = a;
  __syncthreads();
  if (run == 0 && c < p.H) {
    a = 0.f;
#pragma unroll
    for (int w = 0; w < RUNS; ++w) a += s[w][col];
    p.out[blockIdx.y][c] = a;
  }
  // (not sooner: CTAs of the next call's kernel that come while these hold registers do not all find their place)
  pdl_launch_dependents();
}

// (half the columns to a CTA where SMs would have none otherwise: the prenorm's 4096 x 2048 17.1 -> 16.1 us)
template <bool ODD>
cudaError_t launch_sums(const SumDev& q, int sums, cudaStream_t s) {
  const int groups = (q.H + 31) / 32;
  if (q.rows <= 64) MOE_LAUNCH((k_sum_rows<128, 32, ODD>), dim3(groups, sums), dim3(128), 0, s, q);
  else if (groups * sums >= 152) MOE_LAUNCH((k_sum_rows<512, 32, ODD>), dim3(groups, sums), dim3(512), 0, s, q);
  else MOE_LAUNCH((k_sum_rows<512, 16, ODD>), dim3((q.H + 15) / 16, sums), dim3(512), 0, s, q);
  return cudaGetLastError();
}

template <typename T, int NV, int KIND, bool RING, int THREADS, bool ODD, bool FAST = false>
cudaError_t launch_one(NormDev p, int most, int* grid, cudaStream_t s) {
  if constexpr (RING && !FAST && !ODD)
    if (p.H % (32 * kElems) == 0 && p.stream[S_DH] && (KIND == N_PRE || (p.post_w && p.stream[S_DOUT])))
      return launch_one<T, NV, KIND, RING, THREADS, ODD, true>(p, most, grid, s);
  static int known[64] = {};
  auto kernel = k_norm_grad<T, NV, KIND, RING, THREADS, FAST, ODD>;
  const int regs = norm_regs(kernel, known);
  if (!regs) return cudaErrorInvalidValue;
  const NormShape q = norm_shape<T>(p, regs, NV * (16 / (int)sizeof(T)), most, RING);
  if constexpr (RING)
    if (!p.stages) return launch_one<T, NV, KIND, false, THREADS, ODD>(p, most, grid, s);
  *grid = q.grid;
  MOE_LAUNCH(kernel, dim3(q.grid), dim3(q.threads), q.smem, s, p);
  return cudaGetLastError();
}

template <typename T, int KIND, bool ODD>
cudaError_t launch_kind(const NormDev& p, int most, int* grid, cudaStream_t s) {
  constexpr int N = 16 / sizeof(T), NV = kElems / N;
  const int elems = norm_elems(p.H, N);
  if constexpr (!ODD && KIND == N_PRE)
    if (elems > 256 * kElems && elems <= kTwoCtas * kElems) return launch_one<T, NV, KIND, true, kTwoCtas, ODD>(p, most, grid, s);
  return elems > 512 * kElems ? launch_one<T, long_elems(ODD) / N, KIND, false, long_threads(ODD), ODD>(p, most, grid, s)
                              : launch_one<T, NV, KIND, true, 512, ODD>(p, most, grid, s);
}
template <typename T, bool ODD>
cudaError_t launch_width(const NormDev& p, int kind, int most, int* grid, cudaStream_t s) {
  return kind == N_PRE ? launch_kind<T, N_PRE, ODD>(p, most, grid, s)
         : kind == N_POST ? launch_kind<T, N_POST, ODD>(p, most, grid, s)
                          : launch_kind<T, N_FULL, ODD>(p, most, grid, s);
}

}  // namespace

// Rows of partial sums of a gradient: its CTAs at most (two of 256 threads to an SM).
int norm_grad_rows(int T, int H) {
  const int threads = norm_threads(H, kElems);
  return std::min(T, 152 * std::max(norm_ctas(threads, 128), threads <= kTwoCtas ? 2 : 1));
}

cudaError_t launch_norm_grad(const NormArgs& a, cudaStream_t s) {
  NormDev p = norm_dev(a);
  p.part = static_cast<float*>(a.workspace);
  p.sum_post = a.d_post_w != nullptr;
  p.sum_next = a.d_next_w != nullptr;
  p.sum_gate = a.rule.gate == MOE_GATE_CHANNEL && a.d_gate;
  const int kind = !a.y ? N_PRE : a.rule.gate == MOE_GATE_FULL ? N_FULL : N_POST;
  const bool odd = (long)a.H * (a.bf16 ? 2 : 4) % 16 != 0;
  const int most = norm_grad_rows(a.T, a.H);
  int rows = 0;
  cudaError_t e;
  if (a.bf16) e = odd ? launch_width<__nv_bfloat16, true>(p, kind, most, &rows, s) : launch_width<__nv_bfloat16, false>(p, kind, most, &rows, s);
  else e = odd ? launch_width<float, true>(p, kind, most, &rows, s) : launch_width<float, false>(p, kind, most, &rows, s);
  if (e != cudaSuccess || !(p.sum_post || p.sum_next || p.sum_gate)) return e;
  SumDev q = {};
  int sums = 0;
  const size_t plane = (size_t)rows * norm_pitch(a.H);
  float* const out[3] = {a.d_post_w, a.d_next_w, p.sum_gate ? static_cast<float*>(a.d_gate) : nullptr};
  for (int i = 0; i < 3; ++i)
    if (out[i]) {
      q.part[sums] = p.part + i * plane;
      q.out[sums++] = out[i];
    }
  q.rows = rows;
  q.H = a.H;
  q.n = a.bf16 ? 8 : 4;
  return odd ? launch_sums<true>(q, sums, s) : launch_sums<false>(q, sums, s);
}

}  // namespace moe
