// Norms before and after a block, with the block's gate and residual scale, and their gradients.
//
//   prenorm    h = x r w,  r = (mean x^2 + eps)^-1/2
//   postnorm   n = y r_y,  v = n post_w (v = y without a norm),  out = res_scale x + scale G v,
//              h = out r_o next_w (the next block's prenorm, from the unrounded out)
//   gradients  of a norm n = x r with d_n = g:  d_x = r (g - n mean(g n))
//              D = d_out + that of h at out;  d_x = res_scale D,  d_v = scale G D,  d_G = scale D v,
//              d_post_w = sum_t d_v n,  d_next_w = sum_t d_h out r_o,  d_y from d_v post_w
//
// Everything is fp32 between the loads and the one rounding of each result.  The gradients recompute the
// forward pass from x and y: statistics kept by the forward pass would save no bytes, and a rounded out
// would not be the one that the norm saw.
//
// Bound by HBM.  The CTAs are persistent and take every gridDim-th row; a ring of rows in shared memory is filled by
// bulk copies several rows ahead, so that the sums over a row wait for no load.  A row is looked at twice, with one
// barrier between: every sum that it needs follows from sums of products of its inputs.  With c = y post_w gate,
// e = d_h next_w, b = scale r_y (times a token's gate):
//   sum out^2 = res^2 sum x^2 + 2 res b sum x c + b^2 sum c^2,   sum out e = res sum x e + b sum c e,
//   sum g n (for d_y) = scale r_y (sum d_out c + r_o sum e c - r_o^2 m sum out c),  m = mean(e out r_o)
// (A row whose residual and branch cancel, so that the first of these lost digits, is summed again from out: parts_fail.)
// The weights' gradients are
// sums over rows: a CTA keeps those of its rows in registers, writes one fp32 row of partial sums, and a second
// kernel adds the CTAs' rows in their order.
// Beside the bytes, instructions bound it: with the weights loaded and widened in every row and the calls' forms
// told apart there, 16384 x 4096 took 35 of them for an element.  So a thread keeps its columns' weights in
// registers (the norm's after the block times a gate by channels as one factor), works on pairs (f32x2), and
// the gradients of that norm's weight and of such a gate are one sum times the other factor.
// Rows that are no whole 16-byte units are taken in the aligned units that hold them, which every stream and result of
// a row share; a CTA's rows all begin at the same place in a unit (the grid is a multiple of 8), so that a
// thread's columns stay the same.  Where two rows do not fit into a ring, they are read from memory each time.
#pragma once
#include <algorithm>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_vec.cuh"

namespace moe {

// N consecutive values of a weight (or gate) vector of fp32 or bf16
template <int N>
__device__ __forceinline__ void load_w(const void* w, bool f32, size_t i, float (&f)[N]) {
  constexpr int WB = N * 2;  // bytes of N bf16
  if (f32) {
    constexpr int WF = N * 4 >= 16 ? 16 : N * 4;
    using V = typename Word<WF>::type;
    constexpr int per = WF / 4;
#pragma unroll
    for (int q = 0; q < N / per; ++q) {
      float g[per];
      widen<float, WF>(reinterpret_cast<const V*>(static_cast<const float*>(w) + i)[q], g);
#pragma unroll
      for (int c = 0; c < per; ++c) f[q * per + c] = g[c];
    }
  } else {
    using V = typename Word<WB>::type;
    widen<__nv_bfloat16, WB>(*reinterpret_cast<const V*>(static_cast<const uint16_t*>(w) + i), f);
  }
}

__device__ __forceinline__ void sts_one(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_one(uint32_t a, __nv_bfloat16 v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(__bfloat16_as_ushort(v)) : "memory");
}

__device__ __forceinline__ float load_one(const void* w, bool f32, size_t i) {
  return f32 ? static_cast<const float*>(w)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(w)[i]);
}

// exp(-a), a >= 0.  For bf16 rows in a few instructions: 2^t for the rounded product t = -a log2(e), times 1 + r ln(2) for
// what that rounding left (a fused multiply-add gives a product's rounding error exactly; log2(e) in two parts).  Off by 2^-22;
// 0 below 2^-126.  NEAR leaves r out and is off by 2^-22 + 1.3 a 2^-24.
template <typename T, bool NEAR>
__device__ __forceinline__ float exp_minus(float a) {
  if constexpr (sizeof(T) == 4) return expf(-a);
  constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;
  float e;
  if constexpr (NEAR) {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-a * kLog2e));
    return e;
  }
  asm("min.NaN.f32 %0, %0, 0f43000000;" : "+f"(a));  // (128, where e is 0: an infinite a would have no r)
  const float t = -a * kLog2e, r = fmaf(-a, kRest, fmaf(-a, kLog2e, -t));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return fmaf(e, r * kLn2, e);
}
// A quotient by a number from 1 to 2.  (bf16 rows: off by two units instead of a half)
template <typename T>
__device__ __forceinline__ float quotient(float a, float b) {
  if constexpr (sizeof(T) == 4) return a / b;
  return __fdividef(a, b);
}
// A gate's sigmoid s and its slope s (1 - s).  With e = exp(-|z|) and q = 1 / (1 + e), q and e q are the sigmoids of |z| and
// -|z|, and their product the slope: nothing cancels where the gate is nearly open.
template <typename T>
__device__ __forceinline__ float2 sigmoid(float z) {
  const float e = exp_minus<T, false>(fabsf(z)), q = quotient<T>(1.0f, 1.0f + e);
  return make_float2(z >= 0.0f ? q : e * q, e * q * q);
}
// Both in one number w, for gates that wait in registers: the smaller of s and 1 - s, negative where that is 1 - s.
template <typename T>
__device__ __forceinline__ float gate_word(float z) {
  const float e = exp_minus<T, true>(fabsf(z));
  return copysignf(quotient<T>(e, 1.0f + e), -z);
}
__device__ __forceinline__ float word_gate(float w) { return w + __int_as_float(__float_as_int(w) >> 31 & 0x3f800000); }
__device__ __forceinline__ float word_slope(float w) { return fmaf(-w, w, fabsf(w)); }

// The sums of K <= 8 values over the CTA, in every thread, in a fixed order, and a barrier of its threads.  s: 8 floats a warp.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) {
    __syncwarp();  // (the row before may be overwritten behind this: a shuffle alone orders no reads)
    return;
  }
  if (lane == 0) {
    float* at = s + (threadIdx.x >> 5) * 8;
#pragma unroll
    for (int k = 0; k < K; ++k) at[k] = v[k];
  }
  __syncthreads();
  // lane l: value l % 8 of every fourth warp
  float a = 0.f;
  for (int w = lane >> 3; w < warps; w += 4) a += s[w * 8 + (lane & 7)];
  a += __shfl_xor_sync(0xffffffffu, a, 8);
  a += __shfl_xor_sync(0xffffffffu, a, 16);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, a, k);
}
__device__ __forceinline__ float flat(float2 a) { return a.x + a.y; }

// Whether a row's sums in parts are not to be trusted, and it is summed again from out.  E = p + q + 2 c with p, q >= 0
// and q = b^2 cc: each part is off by some 2^-22 of p + q, which an E of an eighth of it turns into 2^-19 at most.
// Nor are they where y post_w gate, without r_y, left the range whose squares fp32 holds, although out did not.
__device__ __forceinline__ bool parts_fail(float p, float q, float e, float b, float cc) {
  return !(e >= 0.125f * (p + q) && p + q < 1e38f) || (cc < 1e-30f && b * b > 1e8f);
}

enum { S_X = 0, S_Y, S_DOUT, S_DH, S_GATE, S_MAX };

struct NormDev {
  const void* stream[S_MAX];  // [T][H], of the activations' type but for the gate (null: none)
  const void *post_w, *gate, *next_w;
  void *out, *h;
  void *d_x, *d_y, *d_gate;
  float* part;       // partial sums: [3][gridDim.x][norm_pitch(H)] of d_post_w, d_next_w, d_gate
  int T, H;
  float inv_h, eps, scale, res_scale;
  int gate_kind;     // MOE_GATE_*
  bool sigmoid, w_f32, gate_f32;
  bool sum_post, sum_next, sum_gate;
  bool gate_ring;    // a full gate of the activations' type: comes through the ring too
  int stages;        // rows of the ring
  uint32_t pitch;    // bytes of a stream's row in it
  int streams;
  int* status;
};

// The rows of a CTA, in turn, NV units of 16 bytes to a thread (units i, i + blockDim, ...): from a ring in shared
// memory (RING) or from memory.  A unit is N elements, C2 pairs; elements outside the row are 0.  FULL_ROWS: every
// thread has all of its units.  ODD: rows begin `lead` elements into their first unit.
template <typename T, int NV, bool RING, bool FULL_ROWS, bool ODD>
struct Rows {
  static constexpr int N = 16 / sizeof(T), C2 = N / 2;
  const NormDev& p;
  uint32_t buf, bars;
  volatile int* abort;
  int lead, units, behind;       // units of a row, elements of its last unit behind it
  int k, stage;                  // rows so far; the present one's place
  uint32_t phase, first;         // first: this thread's first unit in the present stage
  size_t at;                     // element offset of the present row
  bool ok;
  float token;                   // the next row's gate
  int place[S_MAX];              // of a stream among those of a stage
  uint32_t in[ODD ? NV : 1];     // which elements of a unit are in the row: the same in every row, so found once

  __device__ __forceinline__ Rows(const NormDev& q, uint8_t* smem)
      : p(q), lead(0), behind(0), k(0), stage(0), phase(0), first(0), at(0), ok(true), token(1.0f) {
    if (ODD) lead = (int)((size_t)blockIdx.x * p.H % N);
    units = (lead + p.H + N - 1) / N;
    if constexpr (ODD) {
      behind = units * N - lead - p.H;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        in[i] = 0;
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (inside(i, c)) in[i] |= 1u << c;
      }
    }
    if constexpr (RING) {
      abort = reinterpret_cast<volatile int*>(smem);
      bars = smem_u32(smem) + 16;
      buf = smem_u32(smem) + 128;
      int n = 0;
#pragma unroll
      for (int s = 0; s < S_MAX; ++s) place[s] = p.stream[s] && (s != S_GATE || p.gate_ring) ? n++ : 0;
      if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < p.stages; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
      }
    }
  }
  __device__ __forceinline__ int unit(int i) const { return threadIdx.x + i * blockDim.x; }
  __device__ __forceinline__ bool has(int i) const { return FULL_ROWS || unit(i) < units; }
  __device__ __forceinline__ int column(int i) const { return unit(i) * N - lead; }  // of a unit's first element
  __device__ __forceinline__ bool inside(int i, int c) const { return !ODD || (unsigned)(column(i) + c) < (unsigned)p.H; }
  __device__ __forceinline__ bool whole(int i) const { return !ODD || in[ODD ? i : 0] == (1u << N) - 1; }
  // The units of row t that a copy takes: first byte and their bytes.
  __device__ __forceinline__ void extent(int t, size_t& from, uint32_t& n) const {
    const size_t row = (size_t)p.H * sizeof(T), begin = (size_t)t * row, end = begin + row;
    from = begin & ~(size_t)15;
    const size_t up = (end + 15) & ~(size_t)15;
    // (nothing behind the tensor is read: last_unit puts in what the copy leaves out)
    const size_t till = !ODD || up <= (size_t)p.T * row ? up : end & ~(size_t)15;
    n = till > from ? (uint32_t)(till - from) : 0;
  }
  __device__ __forceinline__ void issue(int t, int s) {  // (one thread)
    size_t from;
    uint32_t n;
    extent(t, from, n);
    const uint32_t bar = bars + 8 * s;
    mbar_arrive_expect_tx(bar, n * p.streams);
    if (!n) return;
#pragma unroll
    for (int i = 0; i < S_MAX; ++i)
      if (p.stream[i] && (i != S_GATE || p.gate_ring))
        bulk_g2s(buf + (uint32_t)(s * p.streams + place[i]) * p.pitch, static_cast<const uint8_t*>(p.stream[i]) + from, n, bar);
  }
  __device__ __forceinline__ void start() {  // behind a barrier after the constructor
    if (RING && threadIdx.x == 0)
      for (int s = 0; s < p.stages; ++s) {
        const long t = blockIdx.x + (long)s * gridDim.x;
        if (t < p.T) issue((int)t, s);
      }
  }
  __device__ __forceinline__ void open(int t) {
    at = (size_t)t * p.H;
    if constexpr (RING) {
      if (ok) ok = mbar_wait_one(bars + 8 * stage, phase, abort, p.status);
      first = buf + (uint32_t)(stage * p.streams) * p.pitch + threadIdx.x * 16;
      if (ODD && min(p.T - 1 - t, N) * p.H < behind) last_unit();
    }
  }
  // The last rows of a tensor that ends inside a unit: the copy left that unit out, and the thread that looks at
  // it puts it into the ring (the stage is not filled again: the grid has more rows than a unit has elements).
  __device__ __forceinline__ void last_unit() {
    const int u = units - 1;
    if ((int)threadIdx.x != u % (int)blockDim.x) return;
    for (int s = 0, n = 0; s < S_MAX; ++s) {
      if (!p.stream[s] || (s == S_GATE && !p.gate_ring)) continue;
      const uint32_t to = buf + (uint32_t)(stage * p.streams + n++) * p.pitch + u * 16;
      const T* base = static_cast<const T*>(p.stream[s]) + at;
      for (int c = max(0, u * N - lead); c < p.H; ++c) sts_one(to + (c - (u * N - lead)) * (int)sizeof(T), base[c]);
    }
  }
  // Called behind a barrier in every row: the row before has been read by all.
  __device__ __forceinline__ void refill(int t) {
    if constexpr (RING) {
      if (threadIdx.x == 0 && k > 0) {
        const long next = t + (long)(p.stages - 1) * gridDim.x;
        if (next < p.T) issue((int)next, stage == 0 ? p.stages - 1 : stage - 1);
      }
    }
  }
  __device__ __forceinline__ void close() {
    if constexpr (RING) {
      ++k;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    } else {
      ++k;
    }
  }
  __device__ __forceinline__ void drain() {  // a wait gave up: let the copies in flight land before the CTA ends
    if (RING && !ok && threadIdx.x == 0)
      for (int i = 0; i < p.stages; ++i) {
        mbar_wait_drain(bars + 8 * i, 0, 50000000ull);
        mbar_wait_drain(bars + 8 * i, 1, 50000000ull);
      }
  }
  __device__ __forceinline__ uint4 from_memory(int s, int i) const {
    const T* base = static_cast<const T*>(p.stream[s]);
    if (!ODD || at - lead + (size_t)(unit(i) + 1) * N <= (size_t)p.T * p.H)
      return *reinterpret_cast<const uint4*>(base + (at - lead) + (size_t)unit(i) * N);
    float f[N];  // (the tensor ends in this unit)
#pragma unroll
    for (int c = 0; c < N; ++c) f[c] = inside(i, c) ? to_f32(base[at + column(i) + c]) : 0.f;
    return narrow<T, 16>(f);
  }
  __device__ __forceinline__ static void put(float2 (&f)[C2], int e, float v) {  // (e known at compile time)
    if (e & 1) f[e / 2].y = v;
    else f[e / 2].x = v;
  }
  __device__ __forceinline__ static float pick(const float2 (&f)[C2], int e) { return e & 1 ? f[e / 2].y : f[e / 2].x; }
  // (there: false of a stream that the call does not have: zeros, by a predicate rather than by a branch that the
  // loads would wait behind)
  __device__ __forceinline__ void load(int s, int i, float2 (&f)[C2], bool there = true) const {
    uint4 v = make_uint4(0, 0, 0, 0);
    if constexpr (RING) {
      if (there && has(i)) v = lds_v4(first + (uint32_t)place[s] * p.pitch + (uint32_t)(i * blockDim.x) * 16);
    } else {
      if (there && has(i)) v = from_memory(s, i);
    }
    if constexpr (ODD) {
      if (!whole(i)) {  // (few threads)
        uint32_t m[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if constexpr (N == 4) m[w] = 0u - (in[i] >> w & 1u);
          else m[w] = (in[i] >> (2 * w) & 1u) * 0xffffu | (in[i] >> (2 * w + 1) & 1u) * 0xffff0000u;
        }
        v.x &= m[0];
        v.y &= m[1];
        v.z &= m[2];
        v.w &= m[3];
      }
    }
    float g[N];
    widen<T, 16>(v, g);
#pragma unroll
    for (int c = 0; c < N; ++c) put(f, c, g[c]);
  }
  __device__ __forceinline__ void store(void* base, int i, const float2 (&f)[C2]) const {
    if (!has(i)) return;
    float g[N];
#pragma unroll
    for (int c = 0; c < N; ++c) g[c] = pick(f, c);
    T* to = static_cast<T*>(base) + at;
    if (whole(i)) {
      *reinterpret_cast<uint4*>(to + column(i)) = narrow<T, 16>(g);
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (inside(i, c)) {
          if constexpr (sizeof(T) == 4) to[column(i) + c] = g[c];
          else to[column(i) + c] = __float2bfloat16_rn(g[c]);
        }
    }
  }
  // N partial sums of the unit's columns, in a row of them that begins at the row's first unit
  __device__ __forceinline__ void store_part(float* to, int i, const float2 (&f)[C2]) const {
    if (!has(i)) return;
#pragma unroll
    for (int c = 0; c < N; c += 4)
      *reinterpret_cast<float4*>(to + unit(i) * N + c) = make_float4(f[c / 2].x, f[c / 2].y, f[c / 2 + 1].x, f[c / 2 + 1].y);
  }
  // A weight (or gate) of the unit's columns, from element `from` on.
  __device__ __forceinline__ void weight(const void* w, bool f32, size_t from, int i, float2 (&f)[C2]) const {
    float g[N];
#pragma unroll
    for (int c = 0; c < N; ++c) g[c] = 0.f;
    if (has(i)) {
      if constexpr (!ODD) {
        load_w<N>(w, f32, from + column(i), g);
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c)
          if (inside(i, c)) g[c] = load_one(w, f32, from + column(i) + c);
      }
    }
#pragma unroll
    for (int c = 0; c < N; ++c) put(f, c, g[c]);
  }
  // A gate by channels, and its slope (1 without a sigmoid).
  __device__ __forceinline__ void channel_gate(int i, float2 (&g)[C2], float2 (&slope)[C2]) const {
    weight(p.gate, p.gate_f32, 0, i, g);
#pragma unroll
    for (int e = 0; e < C2; ++e) slope[e] = both(1.f);
    if (p.sigmoid)
#pragma unroll
      for (int e = 0; e < C2; ++e) {
        const float2 a = sigmoid<T>(g[e].x), b = sigmoid<T>(g[e].y);
        g[e] = make_float2(a.x, b.x);
        slope[e] = make_float2(a.y, b.y);
      }
  }
  // The factor of the columns after the block: post_w times a gate by channels (1 where there is neither).
  template <bool CHANNELS>
  __device__ __forceinline__ void factor(int i, float2 (&f)[C2]) const {
#pragma unroll
    for (int e = 0; e < C2; ++e) f[e] = both(1.f);
    if (p.post_w) weight(p.post_w, p.w_f32, 0, i, f);
    if (CHANNELS && p.gate_kind == MOE_GATE_CHANNEL) {
      float2 g[C2], slope[C2];
      channel_gate(i, g, slope);
#pragma unroll
      for (int e = 0; e < C2; ++e) f[e] = mul2(f[e], g[e]);
    }
  }
  // A full gate (with a sigmoid as words), its value, and its slope where it has one.  bf16 rows take the near exponential:
  // with the other the gradient of 8192 x 4096 took 122 us instead of 105 (told apart by the gate's type, 107; its forward
  // pass of 2048 x 16384 86 instead of 80).
  __device__ __forceinline__ void full_gate(int i, float2 (&w)[C2]) const {
    if (p.gate_ring) load(S_GATE, i, w);
    else weight(p.stream[S_GATE], p.gate_f32, at, i, w);
    if (p.sigmoid)
#pragma unroll
      for (int e = 0; e < C2; ++e) w[e] = make_float2(gate_word<T>(w[e].x), gate_word<T>(w[e].y));
  }
  __device__ __forceinline__ float2 gate_of(float2 w) const {
    return p.sigmoid ? make_float2(word_gate(w.x), word_gate(w.y)) : w;
  }
  __device__ __forceinline__ static float2 slope_of(float2 w) { return make_float2(word_slope(w.x), word_slope(w.y)); }
  // A token's gate and its slope, loaded a row ahead.
  __device__ __forceinline__ void fetch_token(long t) {
    if (p.gate_kind == MOE_GATE_TOKEN && t < p.T) token = load_one(p.gate, p.gate_f32, t);
  }
  __device__ __forceinline__ float2 token_gate(int t) {
    if (p.gate_kind != MOE_GATE_TOKEN) return both(1.0f);
    const float g = token;
    fetch_token((long)t + gridDim.x);
    return p.sigmoid ? sigmoid<T>(g) : make_float2(g, 1.0f);
  }
};

// What a kernel does: the prenorm, the postnorm, the postnorm with a gate of [T][H].
enum { N_PRE = 0, N_POST, N_FULL };

// Elements of a thread: 16; for few forward rows 8 (a row is over sooner: one of 4096 1.6 us instead of 1.8).
constexpr int kElems = 16;
// ... and threads of a row that 512 of them do not hold (1024 of 16 would not hold the units of 16383 elements).
constexpr int long_elems(bool odd) { return odd ? 24 : kElems; }
constexpr int long_threads(bool odd) { return odd ? 704 : 1024; }
inline int norm_threads(int elems, int per) { return std::max(32, ((elems + per - 1) / per + 31) / 32 * 32); }
// Elements of the units that may hold a row
inline int norm_elems(int H, int n) { return H % n ? H + 2 * n - 2 : H; }
// CTAs of an SM that `regs` registers a thread leave room for
inline int norm_ctas(int threads, int regs) { return std::max(1, std::min(16, 65536 / ((regs + 7) / 8 * 8 * threads))); }

constexpr int kMaxStages = 8;
constexpr size_t kSmemSm = 226 * 1024;

// Rows of the ring of one of `ctas` CTAs, and its bytes
inline int ring_stages(size_t row, int ctas, size_t* bytes) {
  const size_t room = kSmemSm / ctas - 4 * 1024;  // (static shared memory and what the system takes)
  const int n = (int)std::min<size_t>(kMaxStages, (room - 128) / row);
  *bytes = n < 2 ? 0 : 128 + n * row;
  return n < 2 ? 0 : n;
}

// Sizes of a launch: ring, CTAs and threads.
struct NormShape {
  int threads, grid;
  size_t smem;
};
template <typename T>
NormShape norm_shape(NormDev& p, int regs, int per, int most, bool ring) {
  constexpr int N = 16 / sizeof(T);
  NormShape q;
  q.threads = norm_threads(norm_elems(p.H, N), per);
  int ctas = norm_ctas(q.threads, regs);
  q.smem = 0;
  p.gate_ring = p.gate_ring && ring;
  p.streams = 0;
  for (int i = 0; i < S_MAX; ++i) p.streams += p.stream[i] && (i != S_GATE || p.gate_ring);
  p.pitch = (uint32_t)((norm_elems(p.H, N) + N - 1) / N * 16);
  p.stages = 0;
  // (few CTAs with a ring rather than many without; rows that come about one to a CTA need none)
  if (ring && p.T > 152 * ctas)
    for (int c = ctas;; c /= 2) {
      p.stages = ring_stages((size_t)p.pitch * p.streams, c, &q.smem);
      if (p.stages) ctas = c;
      if (p.stages || c == 1) break;
    }
  q.grid = std::min(std::min(p.T, most), 152 * ctas);
  if (q.grid < p.T && q.grid >= 8) q.grid &= ~7;  // (a CTA's rows begin at the same place in a unit)
  return q;
}
// Registers of a kernel, and its shared memory raised, once for each device.
template <typename K>
int norm_regs(K kernel, int (&known)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && known[dev]) return known[dev];
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemSm - 4 * 1024) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) known[dev] = a.numRegs;
  return a.numRegs;
}

NormDev norm_dev(const NormArgs& a);

}  // namespace moe
