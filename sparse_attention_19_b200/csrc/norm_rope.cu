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
// What cannot be done without is HBM traffic (2 bytes read and 1 or 2 written per element;
// gradient: 4 read, 2 written).  At these widths it sets the pace only if the arithmetic stays
// below ~70 issued instructions per 8 elements: the bf16 form and the gradient come to 0.86 and
// 0.72 of the copy rate, e4m3 (whose kernel's comment has the reason) to 0.62.  So:
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

constexpr int kThreads = 256;
// Blocks of an SM that the registers of the bf16 kernel are to allow: more rows in flight for
// rows of few slots (the layer norm's second sum would spill there), fewer for rows of many.
constexpr int resident(int slots, bool layer) { return slots > 6 ? 1 : slots > 4 || layer ? 2 : 3; }
// The same for the e4m3 kernel, whose barrier per step other blocks have to fill.
constexpr int resident_e4m3(int slots, bool layer) { return slots > 6 ? 1 : slots > 4 ? 2 : layer ? 3 : 4; }
constexpr float kAmaxFloor = 1e-30f;           // an all-zero token keeps a positive scale

struct Vec8 {
  float2 v[4];
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// max(|m|, |x|, |y|), NaN if one of them is.
__device__ __forceinline__ float max_abs(float m, float x, float y) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(x), "f"(y));
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
// FULL rows fill every slot of every lane, the rotated range lies at one end of the row and
// the norm covers all or none of it and of the rest: then nothing is checked per vector
// (8192 x 64 x 128 to e4m3: 57 us with the checks, 53 without).
template <int G, int NP, int NM, bool FULL>
struct Slots {
  static constexpr int kN = 2 * NP + NM;
  int v[FULL ? 1 : kN];      // -1: none
  int pair0, main0;          // FULL: first pair and first other vector of this lane
  bool pair_normed, main_normed;
  int norm_dim;
  __device__ __forceinline__ Slots(const NormRopeParams& p, int lane) {
    const int nv = p.D / 8;
    const int V = p.n_freq ? p.n_freq / 8 : min(G * NP, nv / 2), rs = p.rot_start / 8;
    norm_dim = p.norm_dim;
    if constexpr (FULL) {
      pair0 = rs + lane;
      main0 = lane + (rs == 0 ? 2 * V : 0);
      pair_normed = p.norm_dim > p.rot_start;
      main_normed = p.norm_dim > (rs == 0 ? 16 * V : 0);
    } else {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const int i = n * G + lane;
        v[2 * n] = i < V ? rs + i : -1;
        v[2 * n + 1] = i < V ? rs + V + i : -1;
      }
#pragma unroll
      for (int n = 0; n < NM; ++n) {
        int i = n * G + lane;
        if (i >= rs) i += 2 * V;
        v[2 * NP + n] = i < nv ? i : -1;
      }
    }
  }
  static bool full(const NormRopeParams& p) {
    const int nv = p.D / 8, V = p.n_freq ? p.n_freq / 8 : (G * NP < nv / 2 ? G * NP : nv / 2);
    const int rs = p.rot_start / 8, rest = nv - 2 * V;
    if (V != G * NP || rest != G * NM || (rs != 0 && rs != rest)) return false;
    return p.norm_dim == 0 || p.norm_dim == p.D || (rest > 0 && p.norm_dim == 8 * (rs == 0 ? 2 * V : rest));
  }
  __device__ __forceinline__ int vec(int n) const {
    if constexpr (FULL) return n >= 2 * NP ? main0 + (n - 2 * NP) * G : pair0 + (n / 2 + (n % 2) * NP) * G;
    else return v[n];
  }
  __device__ __forceinline__ bool has(int n) const { return FULL || vec(n) >= 0; }
  // Whether the vector is normalised (norm_dim is 0 without a norm).
  __device__ __forceinline__ bool normed(int n) const {
    if constexpr (FULL) return n >= 2 * NP ? main_normed : pair_normed;
    else return (unsigned)(vec(n) * 8) < (unsigned)norm_dim;
  }
  // Vector n of a row; a group without a row was given an address that can be read.
  __device__ __forceinline__ uint4 load(const uint4* src, int n, bool here) const {
    if constexpr (FULL) return __ldg(src + vec(n));
    else return here && has(n) ? __ldg(src + vec(n)) : make_uint4(0, 0, 0, 0);
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

// x -> xhat = (x - mean) / std over the norm_dim leading columns of a row held by G lanes;
// returns 1/std.  Columns behind them stay as they are.
template <int G, bool LAYER, int N, typename S>
__device__ __forceinline__ float normalise(const NormRopeParams& p, Vec8 (&x)[N], const S& slots) {
  if (p.norm == DSA_NORM_NONE) return 1.f;
  if constexpr (LAYER) {
    float2 s = both(0.f);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (slots.normed(n))
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fadd2(s, x[n].v[e]);
    const float2 nm = both(-group_sum<G>(s.x + s.y) * p.inv_norm_dim);
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (slots.normed(n))
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n].v[e] = fadd2(x[n].v[e], nm);
  }
  float2 q = both(0.f);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (slots.normed(n))
#pragma unroll
      for (int e = 0; e < 4; ++e) q = ffma2(x[n].v[e], x[n].v[e], q);
  const float rstd = rsqrtf(group_sum<G>(q.x + q.y) * p.inv_norm_dim + p.eps);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (slots.normed(n))
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
template <bool LAYER, typename S>
__device__ __forceinline__ void scale8(const NormRopeParams& p, Vec8& z, const S& slots, int n, const float* w) {
  if (!slots.normed(n)) return;
  const int vec = slots.vec(n);
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
struct Row {
  int tok, h;
  bool here;                // whether the group has a row in this step (else: the step's first token)
  __device__ __forceinline__ const uint4* source(const NormRopeParams& p) const {
    const int b = p.div_l(tok), l = tok - b * p.L;
    return reinterpret_cast<const uint4*>(p.x + b * p.stride_b + l * p.stride_l + h * p.stride_h);
  }
  // Vector offset in a contiguous [tokens, H, D] tensor.
  __device__ __forceinline__ size_t offset(const NormRopeParams& p) const {
    return ((size_t)tok * p.H + h) * (p.D / 8);
  }
};
struct Walk {
  int span, step, steps;    // steps: of this span
  int tok0, ntok;           // of the span
  __device__ __forceinline__ void enter(const NormRopeParams& p, int s) {
    span = s;
    step = 0;
    tok0 = s * p.span_tokens;
    ntok = min(p.span_tokens, p.n_tokens - tok0);
    steps = p.parts > 1 ? ntok * p.parts : (ntok + p.tokens_per_step - 1) / p.tokens_per_step;
  }
  // Tokens of a step of whole tokens: the first (in the span) and how many.
  __device__ __forceinline__ int first(const NormRopeParams& p) const { return step * p.tokens_per_step; }
  __device__ __forceinline__ int count(const NormRopeParams& p) const { return min(p.tokens_per_step, ntok - first(p)); }
  // The row of the group that holds head h_in of the step's token tl_in (whole tokens), or
  // the group-th of `groups` heads (part of a token).
  __device__ __forceinline__ Row row(const NormRopeParams& p, int tl_in, int h_in, int group, int groups) const {
    Row r;
    if (p.parts == 1) {
      r.here = tl_in < count(p);
      r.tok = tok0 + first(p) + (r.here ? tl_in : 0);
      r.h = r.here ? h_in : 0;
    } else {
      const int tl = p.div_parts(step), h = (step - tl * p.parts) * groups + group;
      r.here = h < p.H;
      r.tok = tok0 + tl;
      r.h = r.here ? h : 0;
    }
    return r;
  }
};

// amax / 448 and y / scale, each as a product with a reciprocal of two floats whose sum is off
// by less than 2^-44 of itself.  The product's one rounding then gives the rounded quotient
// unless that lies so close to the middle of two floats, which no fp32 value over 448 and no bf16
// value over an fp32 one does: a quotient on the border of two codes stays there.  (The
// bare product with one float crosses it for 1 in 1000 pairs of bf16 significands.  Above
// amax = 2^118 the second float is subnormal and the sum off by up to 2^-31: exact borders stay.)
// Infinities take no second float (inf - inf, 0 * inf): with an infinite scale, finite
// values become 0 and the infinite ones NaN.
__device__ __forceinline__ float scale_of(float amax) {
  constexpr float hi = 1.f / 448.f, lo = (float)(1.0 / 448.0 - (double)hi);
  return isinf(amax) ? amax : fmaf(amax, hi, amax * lo);
}
struct Reciprocal {
  float2 hi, lo;
};
__device__ __forceinline__ Reciprocal reciprocal(float scale) {
  float hi;
  asm("rcp.approx.f32 %0, %1;" : "=f"(hi) : "f"(scale));
  return {both(hi), both(isinf(scale) ? 0.f : fmaf(-scale, hi, 1.f) * hi)};
}

__device__ __forceinline__ uint2 to_e4m3(const Vec8& y, const Reciprocal& r) {
  uint32_t code[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    code[e] = __nv_cvt_float2_to_fp8x2(ffma2(y.v[e], r.hi, fmul2(y.v[e], r.lo)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// bf16 output.  Persistent blocks; while a step is computed the next one's rows are in
// flight, and one barrier per span completes its angles.  Bound by HBM: 0.86-0.90 of the copy
// rate at 4096 x 128 x 192 (72 us; one step per block and nothing in flight behind it 147 us).
template <int G, int NP, int NM, bool FULL, bool LAYER>
__global__ void __launch_bounds__(kThreads, resident(2 * NP + NM, LAYER)) norm_rope_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM, FULL>;
  constexpr int N = S::kN, kGroups = kThreads / G;
  extern __shared__ __align__(16) float smem[];
  const int table = p.span_tokens * p.n_freq;
  float* w = smem + 4 * table;                           // behind two buffers of cos and sin
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int tl_group = p.div_h(group), h_group = group - tl_group * p.H;
  const S slots(p, lane);
  griddep_launch_dependents();
  griddep_wait();
  uint4 raw[N];
  Walk q;
  Row r;
  q.enter(p, blockIdx.x);
  auto load = [&]() {
    r = q.row(p, tl_group, h_group, group, kGroups);
    const uint4* src = r.source(p);
#pragma unroll
    for (int n = 0; n < N; ++n)
      raw[n] = slots.load(src, n, r.here);
  };
  load();
  fill_params(p, w);
  if (p.n_freq) fill_angles(p, q.tok0, q.ntok, smem, smem + table);
  __syncthreads();
  for (int buf = 0;;) {
    Vec8 y[N];
#pragma unroll
    for (int n = 0; n < N; ++n) y[n] = unpack8(raw[n]);
    const bool here = r.here;
    uint4* dst = reinterpret_cast<uint4*>(p.out) + r.offset(p);
    const float* cs = smem + buf * 2 * table + (r.tok - q.tok0) * p.n_freq;
    const bool turn = q.step + 1 == q.steps;             // the span ends with this step
    bool more = true;
    if (!turn) {
      ++q.step;
    } else if (q.span + (int)gridDim.x < p.n_spans) {
      q.enter(p, q.span + gridDim.x);
    } else {
      more = false;
    }
    if (more) load();
    normalise<G, LAYER>(p, y, slots);
#pragma unroll
    for (int n = 0; n < N; ++n) scale8<LAYER>(p, y[n], slots, n, w);
    if (p.n_freq)
#pragma unroll
      for (int n = 0; n < NP; ++n)
        if (slots.has(2 * n)) rotate_pair(p, n * G + lane, y[2 * n], y[2 * n + 1], cs, cs + table, 1.f);
    if (here)
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (slots.has(n)) dst[slots.vec(n)] = pack8(y[n]);
    if (!more) break;
    if (turn) {
      buf ^= 1;
      if (p.n_freq) fill_angles(p, q.tok0, q.ntok, smem + buf * 2 * table, smem + buf * 2 * table + table);
      __syncthreads();
    }
  }
}

// e4m3 output.  A step holds whole tokens, a row per group of lanes in registers; its one
// barrier completes the tokens' maxima.  0.62 of the copy rate at 8192 x 64 x 128 (49.6 us among
// other passes, 48.0 with codes from one rounded reciprocal).  No pipe is full there (issue slots
// 61 %, load/store pipe 58 %): nothing is in flight behind a step, so its warps wait for their own
// rows, for weights and angles from shared memory and at the barrier, and the other three blocks of
// the SM cover only part of that.  Weights and angles come from shared memory for every row,
// since holding them in registers costs more in warps (56 registers: four blocks an SM; the
// weights in registers 63-70 us, two rows per group with one weight read 64 us, five blocks 54 us).
template <int G, int NP, int NM, bool FULL, bool LAYER>
__global__ void __launch_bounds__(kThreads, resident_e4m3(2 * NP + NM, LAYER)) norm_rope_e4m3_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM, FULL>;
  constexpr int N = S::kN, kGroups = kThreads / G;
  extern __shared__ __align__(16) float smem[];
  const int table = p.span_tokens * p.n_freq;
  float* w = smem + 4 * table;                           // behind two buffers of cos and sin
  float* amax3 = w + p.norm_dim * (p.b ? 2 : 1);         // three buffers of one value per token
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int tl_group = p.div_h(group), h_group = group - tl_group * p.H;
  const S slots(p, lane);
  griddep_launch_dependents();
  griddep_wait();
  fill_params(p, w);
  for (int t = threadIdx.x; t < p.tokens_per_step; t += kThreads) amax3[t] = kAmaxFloor;
  int buf = 0, a3 = 0;
  Walk q;
  for (int span = blockIdx.x; span < p.n_spans; span += gridDim.x, buf ^= 1) {
    q.enter(p, span);
    const float* cs0 = smem + buf * 2 * table;
    for (; q.step < q.steps; ++q.step) {
      const Row r = q.row(p, tl_group, h_group, 0, kGroups);
      const uint4* src = r.source(p);
      uint4 raw[N];
#pragma unroll
      for (int n = 0; n < N; ++n) raw[n] = slots.load(src, n, r.here);
      if (q.step == 0) {
        if (p.n_freq) fill_angles(p, q.tok0, q.ntok, smem + buf * 2 * table, smem + buf * 2 * table + table);
        __syncthreads();
      }
      Vec8 y[N];
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = unpack8(raw[n]);
      normalise<G, LAYER>(p, y, slots);
#pragma unroll
      for (int n = 0; n < N; ++n) scale8<LAYER>(p, y[n], slots, n, w);
      const float* cs = cs0 + (r.tok - q.tok0) * p.n_freq;
      if (p.n_freq)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.has(2 * n)) rotate_pair(p, n * G + lane, y[2 * n], y[2 * n + 1], cs, cs + table, 1.f);
      float* amax = amax3 + a3 * p.tokens_per_step;
      a3 = a3 == 2 ? 0 : a3 + 1;
      float* amax_next = amax3 + a3 * p.tokens_per_step;
      const int first = q.tok0 + q.first(p);
      // The maximum does not depend on the order, and a NaN wins (also as an integer).
      float m = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max_abs(m, y[n].v[e].x, y[n].v[e].y);
      if (!r.here) m = 0.f;
      const bool one = p.H % (32 / G) == 0;              // every row of the warp is of one token
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < G || one) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
      if ((one ? threadIdx.x % 32 : lane) == 0 && r.here)
        atomicMax(reinterpret_cast<int*>(&amax[r.tok - first]), __float_as_int(m));
      for (int t = threadIdx.x; t < p.tokens_per_step; t += kThreads) amax_next[t] = kAmaxFloor;
      __syncthreads();
      if (threadIdx.x < q.count(p)) p.scale[first + threadIdx.x] = scale_of(amax[threadIdx.x]);
      if (!r.here) continue;
      const Reciprocal by = reciprocal(scale_of(amax[r.tok - first]));
      uint2* dst = reinterpret_cast<uint2*>(p.codes) + r.offset(p);
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (slots.has(n)) dst[slots.vec(n)] = to_e4m3(y[n], by);
    }
  }
}

// e4m3 of tokens with more heads than a block holds: one block per token, the rows
// computed twice (the second time from L2), first for the maximum.
template <int G, int NP, int NM, bool LAYER>
__global__ void __launch_bounds__(kThreads) norm_rope_wide_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM, false>;
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
        y[n] = unpack8(slots.load(src, n, here));
      normalise<G, LAYER>(p, y, slots);
#pragma unroll
      for (int n = 0; n < N; ++n) scale8<LAYER>(p, y[n], slots, n, w);
      if (p.n_freq)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.has(2 * n)) rotate_pair(p, n * G + lane, y[2 * n], y[2 * n + 1], cs, sn, 1.f);
      if (!here) continue;
      if (pass == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max_abs(m, y[n].v[e].x, y[n].v[e].y);
      } else {
        const Reciprocal by = reciprocal(scale_of(amax));
        uint2* dst = reinterpret_cast<uint2*>(p.codes) + ((size_t)tok * p.H + h) * (p.D / 8);
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (slots.has(n)) dst[slots.vec(n)] = to_e4m3(y[n], by);
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
      if (threadIdx.x % 32 == 0) atomicMax(reinterpret_cast<int*>(&amax), __float_as_int(m));
      __syncthreads();
      if (threadIdx.x == 0) p.scale[tok] = scale_of(amax);
    }
  }
}

// Gradient.  Each block keeps the sums for dw and db of its columns in registers over all its
// steps and leaves one partial row; a second kernel adds the partial rows in block
// order, so the result does not depend on timing.  0.72 of the copy rate at 4096 x 64 x 128 (42.6
// us): the running sums take registers (RMS norm: 127), so 16 warps an SM have to cover the loads.
// Two blocks an SM in one wave: twice as many blocks in two waves took 47 us.  The layer norm's
// db takes 32 registers more than the 128 of two blocks an SM leave: it spills 196 bytes (rows that
// do not fill every slot: 248; widths of six to eight slots run one block, <32,2,4> at 255
// registers with 444 bytes), 13.8 us in this kernel and 8.8 in the second for 16382 keys, caches cold.
template <int G, int NP, int NM, bool FULL, bool LAYER>
__global__ void __launch_bounds__(kThreads, (2 * NP + NM) > 4 ? 1 : 2) norm_rope_bwd_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM, FULL>;
  constexpr int N = S::kN, kGroups = kThreads / G;
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
      const Row r = q.row(p, tl_group, h_group, group, kGroups);
      const size_t row = r.offset(p);
      const uint4* src = r.source(p);
      const uint4* gsrc = reinterpret_cast<const uint4*>(p.dy) + row;
      uint4 raw[N], graw[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        raw[n] = make_uint4(0, 0, 0, 0);
        if (slots.normed(n)) raw[n] = slots.load(src, n, r.here);
        graw[n] = slots.load(gsrc, n, r.here);
      }
      Vec8 xh[N], g[N];                         // xhat; dz, then dz w
#pragma unroll
      for (int n = 0; n < N; ++n) {
        xh[n] = unpack8(raw[n]);
        g[n] = unpack8(graw[n]);
      }
      const float rstd = normalise<G, LAYER>(p, xh, slots);
      if (p.n_freq)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.has(2 * n))
            rotate_pair(p, n * G + lane, g[2 * n], g[2 * n + 1], cs0 + (r.tok - q.tok0) * p.n_freq,
                        cs0 + table + (r.tok - q.tok0) * p.n_freq, -1.f);
      float2 s1 = both(0.f), s2 = both(0.f);    // sums of g and of g xhat
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (!r.here || !slots.normed(n)) continue;   // a group without a row adds nothing
        const Vec8 a = load_angles(w + slots.vec(n) * 8);
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
        if (slots.normed(n)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 t = ffma2(xh[n].v[e], s2, g[n].v[e]);
            g[n].v[e] = fmul2(both(rstd), LAYER ? fadd2(t, s1) : t);
          }
        }
        if (r.here && slots.has(n)) dst[slots.vec(n)] = pack8(g[n]);
      }
    }
  }
  if (p.norm == DSA_NORM_NONE) return;
  // Sum the rows of each warp (exchange) and then the warps (shared memory), in a fixed order.
  float* red = smem;                            // [warps][norm_dim]
  constexpr int kWarps = kThreads / 32;
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
        if (threadIdx.x % 32 < G && slots.normed(n))
          *reinterpret_cast<float2*>(red + warp * p.norm_dim + slots.vec(n) * 8 + 2 * e) = t;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.norm_dim; c += kThreads) {
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
#define DSA_TRY_SPLIT(G, NP, NM)                                                                               \
  if (fits(G, NP, NM)) {                                                                                       \
    if (G <= 8 && Slots<G, NP, NM, (G <= 8)>::full(p))                                                         \
      return f(std::integral_constant<int, G>{}, std::integral_constant<int, NP>{},                            \
               std::integral_constant<int, NM>{}, std::integral_constant<bool, (G <= 8)>{});                   \
    return f(std::integral_constant<int, G>{}, std::integral_constant<int, NP>{}, std::integral_constant<int, NM>{}, \
             std::integral_constant<bool, false>{});                                                           \
  }
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
//   span: a block's even share of the tokens, or an even part of it when the angles of the
//         share would take more than 16 KB.
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
  const long long steps = (n + p.tokens_per_step - 1) / p.tokens_per_step, share = (steps + blocks - 1) / blocks;
  long long most = p.n_freq ? 2048LL / ((long long)p.tokens_per_step * p.n_freq) : share;
  if (most < 1) most = 1;
  const long long rounds = (share + most - 1) / most, k = (steps + blocks * rounds - 1) / (blocks * rounds);
  p.span_tokens = p.tokens_per_step * (int)k;
  p.n_spans = (int)((n + p.span_tokens - 1) / p.span_tokens);
  return (unsigned)(p.n_spans < blocks ? p.n_spans : blocks);
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int sms, cudaStream_t stream) {
  if (!p.n_freq) p.rot_start = 0;
  return by_width(p, [&](auto g, auto np, auto nm, auto full) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, NM = decltype(nm)::value;
    constexpr bool FULL = decltype(full)::value;
    const bool layer = p.norm == DSA_NORM_LAYER;
    const size_t params = (size_t)p.norm_dim * (p.b ? 2 : 1);
    constexpr int kGroups = kThreads / G;
    if (!p.codes) {
      const unsigned grid = plan_walk(p, kGroups, sms, sms * resident(2 * NP + NM, layer));
      const size_t smem = ((size_t)p.span_tokens * p.n_freq * 4 + params) * sizeof(float);
      return launch_pdl(layer ? norm_rope_kernel<G, NP, NM, FULL, true> : norm_rope_kernel<G, NP, NM, FULL, false>, dim3(grid),
                        dim3(kThreads), smem, stream, p);
    }
    if (p.H > kGroups)
      return launch_pdl(layer ? norm_rope_wide_kernel<G, NP, NM, true> : norm_rope_wide_kernel<G, NP, NM, false>,
                        dim3(p.n_tokens), dim3(kThreads), (2 * p.n_freq + params) * sizeof(float), stream, p);
    const unsigned grid = plan_walk(p, kGroups, sms, sms * resident_e4m3(2 * NP + NM, layer));
    const size_t smem = ((size_t)p.span_tokens * p.n_freq * 4 + params + 3 * p.tokens_per_step) * sizeof(float);
    return launch_pdl(layer ? norm_rope_e4m3_kernel<G, NP, NM, FULL, true> : norm_rope_e4m3_kernel<G, NP, NM, FULL, false>,
                      dim3(grid), dim3(kThreads), smem, stream, p);
  });
}

int norm_rope_bwd_blocks(int sms) { return sms * kNormRopeBwdBlocksPerSm; }

cudaError_t launch_norm_rope_bwd(NormRopeParams p, int sms, cudaStream_t stream) {
  if (!p.n_freq) p.rot_start = 0;
  int grid = 0;
  const cudaError_t e = by_width(p, [&](auto g, auto np, auto nm, auto full) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, NM = decltype(nm)::value;
    constexpr bool FULL = decltype(full)::value;
    grid = (int)plan_walk(p, kThreads / G, sms, norm_rope_bwd_blocks(sms));
    size_t smem = ((size_t)p.span_tokens * p.n_freq * 4 + p.norm_dim * (p.b ? 2 : 1)) * sizeof(float);
    const size_t red = (size_t)(kThreads / 32) * p.norm_dim * sizeof(float);
    if (red > smem) smem = red;
    return launch_pdl(p.norm == DSA_NORM_LAYER ? norm_rope_bwd_kernel<G, NP, NM, FULL, true>
                                               : norm_rope_bwd_kernel<G, NP, NM, FULL, false>,
                      dim3(grid), dim3(kThreads), smem, stream, p);
  });
  if (e != cudaSuccess || p.norm == DSA_NORM_NONE) return e;
  return launch_pdl(norm_rope_sum_kernel, dim3((p.norm_dim + 31) / 32, p.b ? 2 : 1), dim3(256), 0, stream, p, grid);
}

}  // namespace dsa
