// norm_rope.cu -- the norm of every query or key head and the position rotation in
// one pass, with the output in bf16 or as the indexer reads it (e4m3 and one scale
// per token), and the gradient of the bf16 form.
//
// For head row x (D columns, fp32 arithmetic on bf16 input):
//   z[i] = (x[i] - mean) * r * w[i] + b[i]   for i < norm_dim, z[i] = x[i] behind it;
//          r = 1/sqrt(mean((x - mean)^2) + eps); RMS norm has mean = 0 and no b;
//   y = z with the pairs (z_a, z_b) of [rot_start, rot_start + 2F) turned by
//       pos * inv_freq[j]:  (z_a c - z_b s, z_b c + z_a s).
// e4m3: scale[token] = max(max |y| over the token's heads, 1e-30) / 448,
//       code = rne(y / scale).
// Gradient, with dz the pairs of dy turned back and xhat = (x - mean) r:
//   g = dz w;  dx = r (g - xhat mean(g xhat) [- mean(g): layer norm]),  dx = dz behind
//   norm_dim;  dw = sum over rows of dz xhat,  db = sum of dz.
//
// Both are bound by HBM (2 bytes read and 1 or 2 written per element; gradient: 4 read, 2
// written), but at these widths only if the arithmetic stays below ~70 issued
// instructions per 8 elements, so:
//   * G lanes hold a head row in 16-byte vectors, and a lane holds BOTH vectors of a rotated
//     pair (NP pair slots, NM slots for the columns that are not rotated): the rotation needs no
//     exchange between lanes and every column is normalised once;
//   * arithmetic runs on packed fp32 pairs (two per instruction);
//   * the angles of a block's tokens are computed once (64-bit range reduction, so a
//     position of 2^31 is as exact as a small one) into shared memory while the rows' loads are
//     in flight; all heads of a token share them.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dsa.h"
#include "dsa_internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kBlocksPerSm = 4;                // blocks of 256 threads
constexpr float kAmaxFloor = 1e-30f;           // an all-zero token keeps a positive scale

struct Vec8 {
  float2 v[4];
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// max(m, |x|), NaN if either is.
__device__ __forceinline__ float max_abs(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
  return r;
}

__device__ __forceinline__ Vec8 unpack8(const uint4& u) {
  Vec8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return r;
}

__device__ __forceinline__ uint32_t pack2(float2 a) {
  const __nv_bfloat162 p = __float22bfloat162_rn(a);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint4 pack8(const Vec8& a) {
  return make_uint4(pack2(a.v[0]), pack2(a.v[1]), pack2(a.v[2]), pack2(a.v[3]));
}

// 8 parameters from column c (16-byte aligned in either type).
__device__ __forceinline__ Vec8 load_param8(const void* w, int is_bf16, int c) {
  if (is_bf16) return unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c)));
  Vec8 r;
  const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
  const float4 a = __ldg(p), b = __ldg(p + 1);
  r.v[0] = make_float2(a.x, a.y); r.v[1] = make_float2(a.z, a.w);
  r.v[2] = make_float2(b.x, b.y); r.v[3] = make_float2(b.z, b.w);
  return r;
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Which vectors of a row a lane holds.  Slots 2n and 2n + 1 (n < NP) are the two members
// of pair vector n * G + lane of the rotated range, the other slots its share of the rest.
// Without a rotation the "range" is the row's first vectors, so that no slot is wasted.
template <int G, int NP, int NM>
struct Slots {
  static constexpr int kN = 2 * NP + NM;
  int vec[kN];               // -1: none
  __device__ __forceinline__ Slots(const NormRopeParams& p, int lane) {
    const int nv = p.D / 8;
    const int V = p.n_freq ? p.n_freq / 8 : min(G * NP, nv / 2), rs = p.rot_start / 8;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int i = n * G + lane;
      vec[2 * n] = i < V ? rs + i : -1;
      vec[2 * n + 1] = i < V ? rs + V + i : -1;
    }
#pragma unroll
    for (int n = 0; n < NM; ++n) {
      int i = n * G + lane;
      if (i >= rs) i += 2 * V;
      vec[2 * NP + n] = i < nv ? i : -1;
    }
  }
};

// cos and sin of the tokens [tok0, tok0 + ntok) for every frequency.
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int tok0, int ntok, float* cs, float* sn) {
  for (int x = threadIdx.x; x < ntok * p.n_freq; x += blockDim.x) {
    const int tl = x / p.n_freq, j = x - tl * p.n_freq;
    const int tok = tok0 + tl;
    const int pos = p.positions ? __ldg(p.positions + tok) : p.q_offset + tok - p.div_l(tok) * p.L;
    const double turns = (double)pos * ((double)__ldg(p.inv_freq + j) * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[x] = c;
    sn[x] = s;
  }
}

__device__ __forceinline__ Vec8 load_angles(const float* t) {
  Vec8 r;
  const float4 a = reinterpret_cast<const float4*>(t)[0], b = reinterpret_cast<const float4*>(t)[1];
  r.v[0] = make_float2(a.x, a.y); r.v[1] = make_float2(a.z, a.w);
  r.v[2] = make_float2(b.x, b.y); r.v[3] = make_float2(b.z, b.w);
  return r;
}

// Turns pair vector i (its members a and b) by the token's angles; `sign` -1 turns back.
// Interleaved rows keep a pair in two neighbouring columns of one vector: frequencies
// 8 (i / 2) + 4 (i % 2) .. for a vector i of the range, and likewise for b's.
__device__ __forceinline__ void rotate_pair(const NormRopeParams& p, int i, Vec8& a, Vec8& b, const float* cs,
                                            const float* sn, float sign) {
  if (!p.interleaved) {
    const Vec8 c = load_angles(cs + 8 * i), s = load_angles(sn + 8 * i);
    const float2 plus = both(sign), minus = both(-sign);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = a.v[e], y = b.v[e];
      a.v[e] = ffma2(x, c.v[e], fmul2(fmul2(minus, s.v[e]), y));
      b.v[e] = ffma2(y, c.v[e], fmul2(fmul2(plus, s.v[e]), x));
    }
  } else {
    const int V = p.n_freq / 8;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      Vec8& z = m ? b : a;
      const int j = 4 * (m ? V + i : i);
      const float4 c = *reinterpret_cast<const float4*>(cs + j), s = *reinterpret_cast<const float4*>(sn + j);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = z.v[e];
        const float t = sign * ss[e];
        z.v[e] = make_float2(x.x * cc[e] - x.y * t, x.y * cc[e] + x.x * t);
      }
    }
  }
}

// Whether a vector is normalised (norm_dim is 0 without a norm; no vector: -1).
__device__ __forceinline__ bool is_normed(const NormRopeParams& p, int vec) {
  return (unsigned)(vec * 8) < (unsigned)p.norm_dim;
}

// x -> xhat = (x - mean) / std over the norm_dim leading columns of a row held by G lanes;
// returns 1/std.  Columns behind them stay as they are.
template <int G, bool LAYER, int N>
__device__ __forceinline__ float normalise(const NormRopeParams& p, Vec8 (&x)[N], const int (&vec)[N]) {
  if (p.norm == DSA_NORM_NONE) return 1.f;
  if constexpr (LAYER) {
    float2 s = both(0.f);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (is_normed(p, vec[n]))
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fadd2(s, x[n].v[e]);
    const float2 nm = both(-group_sum<G>(s.x + s.y) * p.inv_norm_dim);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (is_normed(p, vec[n]))
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n].v[e] = fadd2(x[n].v[e], nm);
  }
  float2 q = both(0.f);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (is_normed(p, vec[n]))
#pragma unroll
      for (int e = 0; e < 4; ++e) q = ffma2(x[n].v[e], x[n].v[e], q);
  const float rstd = rsqrtf(group_sum<G>(q.x + q.y) * p.inv_norm_dim + p.eps);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (is_normed(p, vec[n]))
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n].v[e] = fmul2(x[n].v[e], both(rstd));
  return rstd;
}

// Weights (and biases behind them) as fp32 in shared memory, norm_dim each.
__device__ __forceinline__ void fill_params(const NormRopeParams& p, float* w) {
  for (int c = threadIdx.x * 8; c < p.norm_dim; c += blockDim.x * 8) {
    *reinterpret_cast<Vec8*>(w + c) = load_param8(p.w, p.w_bf16, c);
    if (p.b) *reinterpret_cast<Vec8*>(w + p.norm_dim + c) = load_param8(p.b, p.w_bf16, c);
  }
}

// z = xhat w + b.
template <bool LAYER>
__device__ __forceinline__ void scale8(const NormRopeParams& p, Vec8& z, int vec, const float* w) {
  if (!is_normed(p, vec)) return;
  const Vec8 a = load_angles(w + vec * 8);
  if (LAYER && p.b) {
    const Vec8 b = load_angles(w + p.norm_dim + vec * 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) z.v[e] = ffma2(z.v[e], a.v[e], b.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) z.v[e] = fmul2(z.v[e], a.v[e]);
  }
}

// Steps of a block: spans blockIdx.x, blockIdx.x + gridDim.x, ... of span_tokens tokens, each in
// steps of one row per group of lanes: tokens_per_step whole tokens, or part of a token's heads.
struct Walk {
  int span, step, steps;    // steps: of this span
  int tok0, ntok;           // of the span
  int tl, h;                // this group's row: token in the span and head
  int first, n;             // the step's tokens, in the span
  bool here;                // whether this group has a row
  __device__ __forceinline__ void enter(const NormRopeParams& p, int s) {
    span = s;
    step = 0;
    tok0 = s * p.span_tokens;
    ntok = min(p.span_tokens, p.n_tokens - tok0);
    steps = p.parts > 1 ? ntok * p.parts : (ntok + p.tokens_per_step - 1) / p.tokens_per_step;
  }
  __device__ __forceinline__ void place(const NormRopeParams& p, int group, int groups, int tl_group, int h_group) {
    if (p.parts == 1) {
      first = step * p.tokens_per_step;
      n = min(p.tokens_per_step, ntok - first);
      tl = first + tl_group;
      h = h_group;
      here = tl_group < n;
    } else {
      first = tl = p.div_parts(step);
      n = 1;
      h = (step - tl * p.parts) * groups + group;
      here = h < p.H;
    }
    if (!here) { tl = first; h = 0; }
  }
  __device__ __forceinline__ const uint4* source(const NormRopeParams& p) const {
    const int tok = tok0 + tl, b = p.div_l(tok), l = tok - b * p.L;
    return reinterpret_cast<const uint4*>(p.x + b * p.stride_b + l * p.stride_l + h * p.stride_h);
  }
  // Vector offset of the row in a contiguous [tokens, H, D] tensor.
  __device__ __forceinline__ size_t row(const NormRopeParams& p) const {
    return ((size_t)(tok0 + tl) * p.H + h) * (p.D / 8);
  }
};

__device__ __forceinline__ uint2 to_e4m3(const Vec8& y, float2 inv) {
  uint32_t code[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) code[e] = __nv_cvt_float2_to_fp8x2(fmul2(y.v[e], inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// 1/scale; y / scale is computed as y * (1 / scale), a few fp32 steps from the quotient at most.
__device__ __forceinline__ float inv_scale(float amax) { return 1.f / (amax * (1.f / 448.f)); }

// Persistent blocks.  While a step is computed the next one's rows are in flight.  One
// barrier per span completes its angles; e4m3 adds one per step, for the tokens' maxima.
template <int G, int NP, int NM, bool E4M3, bool LAYER>
__global__ void __launch_bounds__(E4M3 ? kMaxThreads : 256, (2 * NP + NM) > 6 ? 1 : E4M3 ? 1 : 2)
norm_rope_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM>;
  constexpr int N = S::kN;
  extern __shared__ __align__(16) float smem[];
  const int table = p.span_tokens * p.n_freq;
  float* w = smem + 4 * table;                           // behind two buffers of cos and sin
  float* amax3 = w + p.norm_dim * (p.b ? 2 : 1);         // three buffers of one value per token (e4m3)
  const int groups = blockDim.x / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int tl_group = p.div_h(group), h_group = group - tl_group * p.H;
  const S slots(p, lane);
  griddep_launch_dependents();
  griddep_wait();
  uint4 raw[N];
  Walk q;
  q.enter(p, blockIdx.x);
  q.place(p, group, groups, tl_group, h_group);
  auto load = [&]() {
    const uint4* src = q.source(p);
#pragma unroll
    for (int n = 0; n < N; ++n)
      raw[n] = q.here && slots.vec[n] >= 0 ? __ldg(src + slots.vec[n]) : make_uint4(0, 0, 0, 0);
  };
  load();
  fill_params(p, w);
  if (p.n_freq) fill_angles(p, q.tok0, q.ntok, smem, smem + table);
  if (E4M3)
    for (int t = threadIdx.x; t < p.tokens_per_step; t += blockDim.x) amax3[t] = kAmaxFloor;
  __syncthreads();
  int buf = 0, a3 = 0;
  for (;;) {
    Vec8 y[N];
#pragma unroll
    for (int n = 0; n < N; ++n) y[n] = unpack8(raw[n]);
    const int tl = q.tl, first = q.first, n_now = q.n, tok_now = q.tok0 + q.first;
    const bool here = q.here;
    const size_t row = q.row(p);
    const float* cs = smem + buf * 2 * table + tl * p.n_freq;
    const float* sn = cs + table;
    // The next step's rows.
    const bool turn = q.step + 1 == q.steps;             // the span ends with this step
    bool more = true;
    if (!turn) {
      ++q.step;
    } else if (q.span + (int)gridDim.x < p.n_spans) {
      q.enter(p, q.span + gridDim.x);
    } else {
      more = false;
    }
    if (more) {
      q.place(p, group, groups, tl_group, h_group);
      load();
    }
    normalise<G, LAYER>(p, y, slots.vec);
#pragma unroll
    for (int n = 0; n < N; ++n) scale8<LAYER>(p, y[n], slots.vec[n], w);
    if (p.n_freq)
#pragma unroll
      for (int n = 0; n < NP; ++n)
        if (slots.vec[2 * n] >= 0) rotate_pair(p, n * G + lane, y[2 * n], y[2 * n + 1], cs, sn, 1.f);
    if constexpr (!E4M3) {
      if (here)
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (slots.vec[n] >= 0) reinterpret_cast<uint4*>(p.out)[row + slots.vec[n]] = pack8(y[n]);
    }
    if (turn && more) {
      buf ^= 1;
      if (p.n_freq) fill_angles(p, q.tok0, q.ntok, smem + buf * 2 * table, smem + buf * 2 * table + table);
    }
    if constexpr (E4M3) {
      float* amax = amax3 + a3 * p.tokens_per_step;
      a3 = a3 == 2 ? 0 : a3 + 1;
      float* amax_next = amax3 + a3 * p.tokens_per_step;
      // The maximum does not depend on the order, and a NaN wins (also as an integer).
      float m = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max_abs(max_abs(m, y[n].v[e].x), y[n].v[e].y);
      if (!here) m = 0.f;
      const bool one = p.H % (32 / G) == 0;              // every row of the warp is of one token
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < G || one) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
      if ((one ? threadIdx.x % 32 : lane) == 0 && here)
        atomicMax(reinterpret_cast<int*>(&amax[tl - first]), __float_as_int(m));
      for (int t = threadIdx.x; t < p.tokens_per_step; t += blockDim.x) amax_next[t] = kAmaxFloor;
      __syncthreads();
      if (threadIdx.x < n_now) p.scale[tok_now + threadIdx.x] = amax[threadIdx.x] / 448.f;
      if (here) {
        const float2 inv = both(inv_scale(amax[tl - first]));
        uint2* dst = reinterpret_cast<uint2*>(p.codes) + row;
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (slots.vec[n] >= 0) dst[slots.vec[n]] = to_e4m3(y[n], inv);
      }
    } else {
      if (turn && more) __syncthreads();
    }
    if (!more) break;
  }
}

// e4m3 of tokens with more heads than a block holds: one block per token, the rows
// computed twice (the second time from L2), first for the maximum.
template <int G, int NP, int NM, bool LAYER>
__global__ void __launch_bounds__(kMaxThreads) norm_rope_wide_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM>;
  constexpr int N = S::kN;
  extern __shared__ __align__(16) float smem[];
  __shared__ float amax;
  float *cs = smem, *sn = smem + p.n_freq, *w = sn + p.n_freq;
  const int groups = blockDim.x / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const S slots(p, lane);
  const int tok = blockIdx.x, b = p.div_l(tok), l = tok - b * p.L;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x == 0) amax = kAmaxFloor;
  fill_params(p, w);
  if (p.n_freq) fill_angles(p, tok, 1, cs, sn);
  __syncthreads();
  float m = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int h0 = 0; h0 < p.H; h0 += groups) {
      const int h = h0 + group;
      const bool here = h < p.H;
      const uint4* src = reinterpret_cast<const uint4*>(p.x + b * p.stride_b + l * p.stride_l + (here ? h : 0) * p.stride_h);
      Vec8 y[N];
#pragma unroll
      for (int n = 0; n < N; ++n)
        y[n] = unpack8(here && slots.vec[n] >= 0 ? __ldg(src + slots.vec[n]) : make_uint4(0, 0, 0, 0));
      normalise<G, LAYER>(p, y, slots.vec);
#pragma unroll
      for (int n = 0; n < N; ++n) scale8<LAYER>(p, y[n], slots.vec[n], w);
      if (p.n_freq)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.vec[2 * n] >= 0) rotate_pair(p, n * G + lane, y[2 * n], y[2 * n + 1], cs, sn, 1.f);
      if (!here) continue;
      if (pass == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max_abs(max_abs(m, y[n].v[e].x), y[n].v[e].y);
      } else {
        const float2 inv = both(inv_scale(amax));
        uint2* dst = reinterpret_cast<uint2*>(p.codes) + ((size_t)tok * p.H + h) * (p.D / 8);
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (slots.vec[n] >= 0) dst[slots.vec[n]] = to_e4m3(y[n], inv);
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (threadIdx.x % 32 == 0) atomicMax(reinterpret_cast<int*>(&amax), __float_as_int(m));
      __syncthreads();
      if (threadIdx.x == 0) p.scale[tok] = amax / 448.f;
    }
  }
}

// Gradient.  Each block keeps the sums for dw and db of its columns in registers over all its
// steps and leaves one partial row; a second kernel adds the partial rows in block
// order, so the result does not depend on timing.
constexpr int kBwdThreads = 256;

template <int G, int NP, int NM, bool LAYER>
__global__ void __launch_bounds__(kBwdThreads, (2 * NP + NM) > 4 ? 1 : 2) norm_rope_bwd_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM>;
  constexpr int N = S::kN, kGroups = kBwdThreads / G;
  extern __shared__ __align__(16) float smem[];
  const int table = p.span_tokens * p.n_freq;
  float* w = smem + 4 * table;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int tl_group = p.div_h(group), h_group = group - tl_group * p.H;
  const S slots(p, lane);
  griddep_launch_dependents();
  griddep_wait();
  Vec8 dw[N], db[LAYER ? N : 1];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dw[n].v[e] = both(0.f);
      if (LAYER) db[n].v[e] = both(0.f);
    }
  fill_params(p, w);
  Walk q;
  int buf = 0;
  for (int span = blockIdx.x; span < p.n_spans; span += gridDim.x, buf ^= 1) {
    q.enter(p, span);
    float* cs0 = smem + buf * 2 * table;
    if (p.n_freq) fill_angles(p, q.tok0, q.ntok, cs0, cs0 + table);
    __syncthreads();
    for (; q.step < q.steps; ++q.step) {
      q.place(p, group, kGroups, tl_group, h_group);
      const size_t row = q.row(p);
      const uint4* src = q.source(p);
      const uint4* gsrc = reinterpret_cast<const uint4*>(p.dy) + row;
      uint4 raw[N], graw[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        raw[n] = graw[n] = make_uint4(0, 0, 0, 0);
        if (q.here && slots.vec[n] >= 0) {
          if (is_normed(p, slots.vec[n])) raw[n] = __ldg(src + slots.vec[n]);
          graw[n] = __ldg(gsrc + slots.vec[n]);
        }
      }
      Vec8 xh[N], g[N];                         // xhat; dz, then dz w
#pragma unroll
      for (int n = 0; n < N; ++n) {
        xh[n] = unpack8(raw[n]);
        g[n] = unpack8(graw[n]);
      }
      const float rstd = normalise<G, LAYER>(p, xh, slots.vec);
      if (p.n_freq)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.vec[2 * n] >= 0)
            rotate_pair(p, n * G + lane, g[2 * n], g[2 * n + 1], cs0 + q.tl * p.n_freq, cs0 + table + q.tl * p.n_freq,
                        -1.f);
      float2 s1 = both(0.f), s2 = both(0.f);    // sums of g and of g xhat
#pragma unroll
      for (int n = 0; n < N; ++n) {
        // a group without a row has dz = 0 but perhaps an infinite 1/std: it adds nothing
        if (!q.here || !is_normed(p, slots.vec[n])) continue;
        const Vec8 a = load_angles(w + slots.vec[n] * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dw[n].v[e] = ffma2(g[n].v[e], xh[n].v[e], dw[n].v[e]);
          if (LAYER) db[n].v[e] = fadd2(db[n].v[e], g[n].v[e]);
          g[n].v[e] = fmul2(g[n].v[e], a.v[e]);
          if (LAYER) s1 = fadd2(s1, g[n].v[e]);
          s2 = ffma2(g[n].v[e], xh[n].v[e], s2);
        }
      }
      if (p.norm != DSA_NORM_NONE) {
        s2 = both(-group_sum<G>(s2.x + s2.y) * p.inv_norm_dim);
        if (LAYER) s1 = both(-group_sum<G>(s1.x + s1.y) * p.inv_norm_dim);
      }
      uint4* dst = reinterpret_cast<uint4*>(p.dx) + row;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (is_normed(p, slots.vec[n])) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t = ffma2(xh[n].v[e], s2, g[n].v[e]);
            g[n].v[e] = fmul2(both(rstd), LAYER ? fadd2(t, s1) : t);
          }
        }
        if (q.here && slots.vec[n] >= 0) dst[slots.vec[n]] = pack8(g[n]);
      }
    }
  }
  if (p.norm == DSA_NORM_NONE) return;
  // Sum the rows of each warp (exchange) and then the warps (shared memory), in a fixed order.
  float* red = smem;                            // [warps][norm_dim]
  constexpr int kWarps = kBwdThreads / 32;
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int what = 0; what < (LAYER ? 2 : 1); ++what) {
    if (what && !p.b) break;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 t = what ? db[LAYER ? n : 0].v[e] : dw[n].v[e];
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) {
          t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
          t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
        }
        if (threadIdx.x % 32 < G && is_normed(p, slots.vec[n]))
          *reinterpret_cast<float2*>(red + warp * p.norm_dim + slots.vec[n] * 8 + 2 * e) = t;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.norm_dim; c += kBwdThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += red[k * p.norm_dim + c];
      p.part[((size_t)what * gridDim.x + blockIdx.x) * p.norm_dim + c] = s;
    }
  }
}

// dw and db: one block per 32 columns; 8 warps each add every 8th partial row, and the
// eight sums are added in warp order.
__global__ void __launch_bounds__(256) norm_rope_sum_kernel(const NormRopeParams p, int n_part) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane, what = blockIdx.y;
  float s = 0.f;
  if (c < p.norm_dim) {
    const float* src = p.part + (size_t)what * n_part * p.norm_dim + c;
#pragma unroll 8
    for (int i = warp; i < n_part; i += 8) s += src[(size_t)i * p.norm_dim];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.norm_dim) {
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    (what ? p.db : p.dw)[c] = s;
  }
}

// Row split for a head of D columns of which 2F are rotated: the fewest lanes whose slots
// hold it (most slots per lane: fewest idle lanes and exchange steps), up to 6 slots.
template <typename Fn>
cudaError_t by_width(const NormRopeParams& p, Fn&& f) {
  const int nv = p.D / 8;
  auto fits = [&](int g, int np, int nm) {
    const int v = p.n_freq ? p.n_freq / 8 : (g * np < nv / 2 ? g * np : nv / 2);
    return v <= g * np && nv - 2 * v <= g * nm;
  };
#define DSA_TRY_SPLIT(G, NP, NM) \
  if (fits(G, NP, NM))           \
  return f(std::integral_constant<int, G>{}, std::integral_constant<int, NP>{}, std::integral_constant<int, NM>{})
  DSA_TRY_SPLIT(4, 1, 0);
  DSA_TRY_SPLIT(4, 1, 2);
  DSA_TRY_SPLIT(4, 1, 4);
  DSA_TRY_SPLIT(8, 1, 2);
  DSA_TRY_SPLIT(32, 1, 2);
  DSA_TRY_SPLIT(32, 2, 4);
#undef DSA_TRY_SPLIT
  return cudaErrorInvalidValue;
}

// Steps and spans for blocks of `groups` rows a step; returns the grid.
//   step: as many whole tokens as a block holds, but with few tokens only as many as spread
//         them over the SMs; or part of a token's heads when a block holds less than one;
//   span: steps whose angles together give every thread of the block one to fill in, as
//         long as each block still gets four spans (their work then evens out), and at
//         most 16 KB of angles.
unsigned plan_walk(NormRopeParams& p, int groups, int sms, int blocks) {
  const long long n = p.n_tokens;
  p.parts = (p.H + groups - 1) / groups;
  p.div_parts = fast_div((uint32_t)p.parts);
  long long t = groups / p.H;
  const long long spread = (n + 2 * sms - 1) / (2 * sms);
  if (t > spread) t = spread;
  const long long table = p.n_freq ? 16384 / (8LL * p.n_freq) : t;
  if (t > table) t = table;
  p.tokens_per_step = t < 1 ? 1 : (int)t;
  long long k = p.n_freq ? 256 / ((long long)p.tokens_per_step * p.n_freq) : 8;
  const long long even = n / (4LL * blocks * p.tokens_per_step);
  if (k > even) k = even;
  p.span_tokens = p.tokens_per_step * (k < 1 ? 1 : (int)k);
  p.n_spans = (int)((n + p.span_tokens - 1) / p.span_tokens);
  return (unsigned)(p.n_spans < blocks ? p.n_spans : blocks);
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int sms, cudaStream_t stream) {
  if (!p.n_freq) p.rot_start = 0;
  return by_width(p, [&](auto g, auto np, auto nm) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, NM = decltype(nm)::value;
    const bool layer = p.norm == DSA_NORM_LAYER;
    const size_t params = (size_t)p.norm_dim * (p.b ? 2 : 1);
    if (p.codes && p.H > kMaxThreads / G)
      return launch_pdl(layer ? norm_rope_wide_kernel<G, NP, NM, true> : norm_rope_wide_kernel<G, NP, NM, false>,
                        dim3(p.n_tokens), dim3(kMaxThreads), (2 * p.n_freq + params) * sizeof(float), stream, p);
    // Twice the threads where that lets a block hold all heads of a token (e4m3).
    const int threads = p.codes && p.H > 256 / G ? kMaxThreads : 256;
    const unsigned grid = plan_walk(p, threads / G, sms, sms * (threads == 256 ? kBlocksPerSm : kBlocksPerSm / 2));
    const size_t smem = ((size_t)p.span_tokens * p.n_freq * 4 + params + 3 * p.tokens_per_step) * sizeof(float);
    auto kern = p.codes ? (layer ? norm_rope_kernel<G, NP, NM, true, true> : norm_rope_kernel<G, NP, NM, true, false>)
                        : (layer ? norm_rope_kernel<G, NP, NM, false, true> : norm_rope_kernel<G, NP, NM, false, false>);
    return launch_pdl(kern, dim3(grid), dim3(threads), smem, stream, p);
  });
}

int norm_rope_bwd_blocks(int sms) { return sms * kNormRopeBwdBlocksPerSm; }

cudaError_t launch_norm_rope_bwd(NormRopeParams p, int sms, cudaStream_t stream) {
  if (!p.n_freq) p.rot_start = 0;
  int grid = 0;
  const cudaError_t e = by_width(p, [&](auto g, auto np, auto nm) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, NM = decltype(nm)::value;
    grid = (int)plan_walk(p, kBwdThreads / G, sms, norm_rope_bwd_blocks(sms));
    size_t smem = ((size_t)p.span_tokens * p.n_freq * 4 + p.norm_dim * (p.b ? 2 : 1)) * sizeof(float);
    const size_t red = (size_t)(kBwdThreads / 32) * p.norm_dim * sizeof(float);
    if (red > smem) smem = red;
    return launch_pdl(p.norm == DSA_NORM_LAYER ? norm_rope_bwd_kernel<G, NP, NM, true>
                                               : norm_rope_bwd_kernel<G, NP, NM, false>,
                      dim3(grid), dim3(kBwdThreads), smem, stream, p);
  });
  if (e != cudaSuccess || p.norm == DSA_NORM_NONE) return e;
  return launch_pdl(norm_rope_sum_kernel, dim3((p.norm_dim + 31) / 32, p.b ? 2 : 1), dim3(256), 0, stream, p, grid);
}

}  // namespace dsa
