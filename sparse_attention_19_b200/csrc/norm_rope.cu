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
constexpr int kNormRopeBlocksPerSm = 4;        // blocks of 256 threads
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

// Mean and 1/std of the norm_dim leading columns of a row held by G lanes.
template <int G, int N>
__device__ __forceinline__ void row_stats(const NormRopeParams& p, const uint4 (&raw)[N], const int (&vec)[N],
                                          float& mean, float& rstd) {
  mean = 0.f;
  rstd = 1.f;
  if (p.norm == DSA_NORM_NONE) return;
  const float inv_n = p.inv_norm_dim;
  if (p.norm == DSA_NORM_LAYER) {
    float2 s = both(0.f);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Vec8 x = unpack8(raw[n]);
      if (vec[n] * 8 < p.norm_dim)                       // a missing vector was loaded as zeros
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fadd2(s, x.v[e]);
    }
    mean = group_sum<G>(s.x + s.y) * inv_n;
  }
  float2 q = both(0.f);
  const float2 nm = both(-mean);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Vec8 x = unpack8(raw[n]);
    if (vec[n] >= 0 && vec[n] * 8 < p.norm_dim)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 d = fadd2(x.v[e], nm);
        q = ffma2(d, d, q);
      }
  }
  rstd = rsqrtf(group_sum<G>(q.x + q.y) * inv_n + p.eps);
}

// z of one vector: normalised (columns below norm_dim), or as it is (zeros for no vector).
__device__ __forceinline__ Vec8 normed8(const NormRopeParams& p, const uint4& raw, int vec, float mean, float rstd) {
  Vec8 z = unpack8(raw);
  if ((unsigned)(vec * 8) < (unsigned)p.norm_dim) {      // norm_dim is 0 without a norm; no vector: -1
    const Vec8 w = load_param8(p.w, p.w_bf16, vec * 8);
    const float2 r = both(rstd);
    if (p.norm == DSA_NORM_LAYER) {
      const float2 nm = both(-mean);
#pragma unroll
      for (int e = 0; e < 4; ++e) z.v[e] = fadd2(z.v[e], nm);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) z.v[e] = fmul2(fmul2(z.v[e], r), w.v[e]);
    if (p.b) {
      const Vec8 bias = load_param8(p.b, p.w_bf16, vec * 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) z.v[e] = fadd2(z.v[e], bias.v[e]);
    }
  }
  return z;
}

__device__ __forceinline__ uint2 to_e4m3(const Vec8& y, float2 inv) {
  uint32_t code[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) code[e] = __nv_cvt_float2_to_fp8x2(fmul2(y.v[e], inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// 1/scale; y / scale is computed as y * (1 / scale), a few fp32 steps from the quotient at most.
__device__ __forceinline__ float inv_scale(float amax) { return 1.f / (amax * (1.f / 448.f)); }

// Persistent blocks over chunks of rows, one row per group of G lanes and chunk.  A chunk is
// tokens_per_block whole tokens, or (bf16 only) `groups` heads of one token.  While a chunk
// is computed the next one's rows are in flight, and its angles are filled in before the
// chunk's one barrier; that barrier also completes the tokens' maxima for e4m3.
template <int G, int NP, int NM, bool E4M3>
__global__ void __launch_bounds__(E4M3 ? kMaxThreads : 256, (2 * NP + NM) > 6 ? 1 : E4M3 ? 1 : 2)
norm_rope_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM>;
  constexpr int N = S::kN;
  extern __shared__ __align__(16) float smem[];
  const int table = p.tokens_per_block * p.n_freq;
  float* amax3 = smem + 4 * table;                       // three buffers of one value per token (e4m3)
  const int groups = blockDim.x / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const S slots(p, lane);
  const int parts = E4M3 ? 1 : (p.H + groups - 1) / groups;   // chunks of a token that fills more than one
  // Chunk -> first token, tokens, this group's token in the chunk and head.
  struct Place { int tok0, ntok, tl, h; bool here; };
  auto place = [&](int ch) {
    Place q;
    if (parts == 1) {
      q.tok0 = ch * p.tokens_per_block;
      q.ntok = min(p.tokens_per_block, p.n_tokens - q.tok0);
      q.tl = p.div_h(group);
      q.h = group - q.tl * p.H;
      q.here = q.tl < q.ntok;
    } else {
      q.tok0 = ch / parts;
      q.ntok = 1;
      q.tl = 0;
      q.h = (ch - q.tok0 * parts) * groups + group;
      q.here = q.h < p.H;
    }
    if (!q.here) q.tl = q.h = 0;                         // (reads the first token's angles, writes nothing)
    return q;
  };
  uint4 raw[N];
  auto load = [&](const Place& q) {
    const int tok = q.tok0 + q.tl, b = p.div_l(tok), l = tok - b * p.L;
    const uint4* src = reinterpret_cast<const uint4*>(p.x + b * p.stride_b + l * p.stride_l + q.h * p.stride_h);
#pragma unroll
    for (int n = 0; n < N; ++n)
      raw[n] = q.here && slots.vec[n] >= 0 ? __ldg(src + slots.vec[n]) : make_uint4(0, 0, 0, 0);
  };
  griddep_launch_dependents();
  griddep_wait();
  int ch = blockIdx.x;
  Place q = place(ch);
  load(q);
  fill_angles(p, q.tok0, q.ntok, smem, smem + table);
  if (E4M3)
    for (int t = threadIdx.x; t < p.tokens_per_block; t += blockDim.x) amax3[t] = kAmaxFloor;
  __syncthreads();
  for (int it = 0, a3 = 0; ch < p.n_chunks; ch += gridDim.x, it ^= 1) {
    const float* cs = smem + it * 2 * table;
    const float* sn = cs + table;
    float* amax = amax3 + a3 * p.tokens_per_block;
    a3 = a3 == 2 ? 0 : a3 + 1;
    float* amax_next = amax3 + a3 * p.tokens_per_block;
    float mean, rstd;
    row_stats<G, N>(p, raw, slots.vec, mean, rstd);
    const size_t row = ((size_t)(q.tok0 + q.tl) * p.H + q.h) * (p.D / 8);   // of the output, in vectors
    Vec8 y[E4M3 ? N : 1];
    auto emit = [&](int n, const Vec8& z) {
      if constexpr (E4M3) y[n] = z;
      else if (q.here && slots.vec[n] >= 0) reinterpret_cast<uint4*>(p.out)[row + slots.vec[n]] = pack8(z);
    };
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      Vec8 a = normed8(p, raw[2 * n], slots.vec[2 * n], mean, rstd);
      Vec8 b = normed8(p, raw[2 * n + 1], slots.vec[2 * n + 1], mean, rstd);
      if (p.n_freq && slots.vec[2 * n] >= 0)
        rotate_pair(p, n * G + lane, a, b, cs + q.tl * p.n_freq, sn + q.tl * p.n_freq, 1.f);
      emit(2 * n, a);
      emit(2 * n + 1, b);
    }
#pragma unroll
    for (int n = 2 * NP; n < N; ++n) emit(n, normed8(p, raw[n], slots.vec[n], mean, rstd));

    const Place now = q;
    if (ch + (int)gridDim.x < p.n_chunks) {
      q = place(ch + gridDim.x);
      load(q);
      float* tab = smem + (it ^ 1) * 2 * table;
      fill_angles(p, q.tok0, q.ntok, tab, tab + table);
    }
    if constexpr (E4M3) {
      // The maximum does not depend on the order, and a NaN wins (also as an integer).
      float m = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max_abs(max_abs(m, y[n].v[e].x), y[n].v[e].y);
      if (!now.here) m = 0.f;
      const bool one = p.H >= 32 / G && p.H % (32 / G) == 0;   // every row of the warp is of one token
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < G || one) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
      if ((one ? threadIdx.x % 32 : lane) == 0 && now.here)
        atomicMax(reinterpret_cast<int*>(&amax[now.tl]), __float_as_int(m));
      for (int t = threadIdx.x; t < p.tokens_per_block; t += blockDim.x) amax_next[t] = kAmaxFloor;
    }
    __syncthreads();
    if constexpr (E4M3) {
      if (threadIdx.x < now.ntok) p.scale[now.tok0 + threadIdx.x] = amax[threadIdx.x] / 448.f;
      if (now.here) {
        const float2 inv = both(inv_scale(amax[now.tl]));
        uint2* dst = reinterpret_cast<uint2*>(p.codes) + row;
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (slots.vec[n] >= 0) dst[slots.vec[n]] = to_e4m3(y[n], inv);
      }
    }
  }
}

// e4m3 of tokens with more heads than a block holds: one block per token, the rows
// computed twice (the second time from L2), first for the maximum.
template <int G, int NP, int NM>
__global__ void __launch_bounds__(kMaxThreads) norm_rope_wide_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM>;
  constexpr int N = S::kN;
  extern __shared__ __align__(16) float smem[];
  __shared__ float amax;
  float *cs = smem, *sn = smem + p.n_freq;
  const int groups = blockDim.x / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const S slots(p, lane);
  const int tok = blockIdx.x, b = p.div_l(tok), l = tok - b * p.L;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x == 0) amax = kAmaxFloor;
  fill_angles(p, tok, 1, cs, sn);
  __syncthreads();
  float m = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int h0 = 0; h0 < p.H; h0 += groups) {
      const int h = h0 + group;
      const bool here = h < p.H;
      const uint4* src = reinterpret_cast<const uint4*>(p.x + b * p.stride_b + l * p.stride_l + (here ? h : 0) * p.stride_h);
      uint4 raw[N];
#pragma unroll
      for (int n = 0; n < N; ++n)
        raw[n] = here && slots.vec[n] >= 0 ? __ldg(src + slots.vec[n]) : make_uint4(0, 0, 0, 0);
      float mean, rstd;
      row_stats<G, N>(p, raw, slots.vec, mean, rstd);
      Vec8 y[N];
#pragma unroll
      for (int n = 0; n < N; ++n) y[n] = normed8(p, raw[n], slots.vec[n], mean, rstd);
      if (p.n_freq)
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.vec[2 * n] >= 0) rotate_pair(p, n * G + lane, y[2 * n], y[2 * n + 1], cs, sn, 1.f);
      if (!here) continue;
      if (pass == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (slots.vec[n] >= 0)
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

// Gradient.  Persistent blocks: each walks its chunks of tokens, keeps the sums for dw
// and db of its columns in registers, and leaves one partial row per block; a second
// kernel adds the partial rows in block order, so the result does not depend on timing.
constexpr int kBwdThreads = 256;

template <int G, int NP, int NM, bool BIAS>
__global__ void __launch_bounds__(kBwdThreads, (2 * NP + NM) > 4 ? 1 : 2) norm_rope_bwd_kernel(const NormRopeParams p) {
  using S = Slots<G, NP, NM>;
  constexpr int N = S::kN, kGroups = kBwdThreads / G;
  extern __shared__ __align__(16) float smem[];
  const int table = p.tokens_per_block * p.n_freq;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const S slots(p, lane);
  griddep_launch_dependents();
  griddep_wait();
  Vec8 dw[N], db[BIAS ? N : 1];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dw[n].v[e] = both(0.f);
      if (BIAS) db[n].v[e] = both(0.f);
    }

  const int n_chunks = (int)(((long long)p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block);
  int buf = 0;
  for (int ch = blockIdx.x; ch < n_chunks; ch += gridDim.x, buf ^= 1) {
    const int tok0 = ch * p.tokens_per_block;
    const int ntok = min(p.tokens_per_block, p.n_tokens - tok0);
    const int rows = ntok * p.H;
    const int steps = (rows + kGroups - 1) / kGroups;
    float* cs = smem + buf * 2 * table;         // two tables: the next chunk's may be filled
    float* sn = cs + table;                     // while slower warps still read this one
    for (int st = 0; st < steps; ++st) {
      const int row = st * kGroups + group;
      const bool here = row < rows;
      const int tl = here ? p.div_h(row) : 0, h = here ? row - tl * p.H : 0;
      uint4 raw[N], graw[N];
      {
        const int tok = tok0 + tl, b = p.div_l(tok), l = tok - b * p.L;
        const uint4* src = reinterpret_cast<const uint4*>(p.x + b * p.stride_b + l * p.stride_l + h * p.stride_h);
        const uint4* gsrc = reinterpret_cast<const uint4*>(p.dy + ((size_t)tok0 * p.H + row) * p.D);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          raw[n] = graw[n] = make_uint4(0, 0, 0, 0);
          if (here && slots.vec[n] >= 0) {
            if (slots.vec[n] * 8 < p.norm_dim) raw[n] = __ldg(src + slots.vec[n]);
            graw[n] = __ldg(gsrc + slots.vec[n]);
          }
        }
      }
      if (st == 0) {
        fill_angles(p, tok0, ntok, cs, sn);
        __syncthreads();
      }
      float mean, rstd;
      row_stats<G, N>(p, raw, slots.vec, mean, rstd);
      if (!here) rstd = 0.f;                    // 1/sqrt(eps) may be infinite
      Vec8 g[N];                                // dz, then dz w
#pragma unroll
      for (int n = 0; n < N; ++n) g[n] = unpack8(graw[n]);
      if (p.n_freq) {
#pragma unroll
        for (int n = 0; n < NP; ++n)
          if (slots.vec[2 * n] >= 0)
            rotate_pair(p, n * G + lane, g[2 * n], g[2 * n + 1], cs + tl * p.n_freq, sn + tl * p.n_freq, -1.f);
      }
      const float2 r2 = both(rstd), nm = both(-mean);
      float2 s1 = both(0.f), s2 = both(0.f);    // sums of g and of g xhat
      if (p.norm != DSA_NORM_NONE) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          if (slots.vec[n] < 0 || slots.vec[n] * 8 >= p.norm_dim) continue;
          const Vec8 x = unpack8(raw[n]), w = load_param8(p.w, p.w_bf16, slots.vec[n] * 8);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 xh = fmul2(fadd2(x.v[e], nm), r2);
            // a row past the end has dz = 0, so it adds nothing
            dw[n].v[e] = ffma2(g[n].v[e], xh, dw[n].v[e]);
            if (BIAS) db[n].v[e] = fadd2(db[n].v[e], g[n].v[e]);
            g[n].v[e] = fmul2(g[n].v[e], w.v[e]);
            s1 = fadd2(s1, g[n].v[e]);
            s2 = ffma2(g[n].v[e], xh, s2);
          }
        }
        const float inv_n = p.inv_norm_dim;
        s2 = both(-group_sum<G>(s2.x + s2.y) * inv_n);
        s1 = both(p.norm == DSA_NORM_LAYER ? -group_sum<G>(s1.x + s1.y) * inv_n : 0.f);
      }
      uint4* dst = reinterpret_cast<uint4*>(p.dx + ((size_t)tok0 * p.H + row) * p.D);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (p.norm != DSA_NORM_NONE && slots.vec[n] * 8 < p.norm_dim) {
          const Vec8 x = unpack8(raw[n]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 xh = fmul2(fadd2(x.v[e], nm), r2);
            g[n].v[e] = fmul2(r2, ffma2(xh, s2, fadd2(g[n].v[e], s1)));
          }
        }
        if (here && slots.vec[n] >= 0) dst[slots.vec[n]] = pack8(g[n]);
      }
    }
  }
  if (p.norm == DSA_NORM_NONE) return;
  // Sum the rows of each warp (exchange) and then the warps (shared memory), in a fixed order.
  float* red = smem;                            // [warps][norm_dim]
  constexpr int kWarps = kBwdThreads / 32;
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int what = 0; what < (BIAS ? 2 : 1); ++what) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 t = what ? db[BIAS ? n : 0].v[e] : dw[n].v[e];
#pragma unroll
        for (int o = 16; o >= G; o >>= 1) {
          t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
          t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
        }
        if (threadIdx.x % 32 < G && slots.vec[n] >= 0 && slots.vec[n] * 8 < p.norm_dim)
          *reinterpret_cast<float2*>(red + warp * p.norm_dim + slots.vec[n] * 8 + 2 * e) = t;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.norm_dim; c += kBwdThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w * p.norm_dim + c];
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

// Tokens per block: what one step holds, spread over the SMs when there are few tokens,
// with at most 16 KB of angles.
int tokens_per_block(const NormRopeParams& p, int rows_per_step, int sms) {
  long long t = rows_per_step / p.H;
  const long long spread = ((long long)p.n_tokens + 2 * sms - 1) / (2 * sms);
  if (t > spread) t = spread;
  const long long table = p.n_freq ? 16384 / (8LL * p.n_freq) : t;
  if (t > table) t = table;
  return t < 1 ? 1 : (int)t;
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams p, int sms, cudaStream_t stream) {
  if (!p.n_freq) p.rot_start = 0;
  return by_width(p, [&](auto g, auto np, auto nm) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, NM = decltype(nm)::value;
    if (p.codes && p.H > kMaxThreads / G)
      return launch_pdl(norm_rope_wide_kernel<G, NP, NM>, dim3(p.n_tokens), dim3(kMaxThreads),
                        (size_t)p.n_freq * 8, stream, p);
    // Twice the threads where that lets a block hold all heads of a token (e4m3).
    const int threads = p.codes && p.H > 256 / G ? kMaxThreads : 256, groups = threads / G;
    p.tokens_per_block = tokens_per_block(p, groups, sms);
    const long long chunks = p.H > groups ? (long long)p.n_tokens * ((p.H + groups - 1) / groups)
                                          : ((long long)p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
    if (chunks >= (1ll << 31) - sms * 8) return cudaErrorInvalidValue;
    p.n_chunks = (int)chunks;
    const long long most = (long long)sms * (threads == 256 ? kNormRopeBlocksPerSm : kNormRopeBlocksPerSm / 2);
    const size_t smem = ((size_t)p.tokens_per_block * p.n_freq * 4 + 3 * p.tokens_per_block) * sizeof(float);
    return launch_pdl(p.codes ? norm_rope_kernel<G, NP, NM, true> : norm_rope_kernel<G, NP, NM, false>,
                      dim3((unsigned)(chunks < most ? chunks : most)), dim3(threads), smem, stream, p);
  });
}

int norm_rope_bwd_blocks(int sms) { return sms * kNormRopeBwdBlocksPerSm; }

cudaError_t launch_norm_rope_bwd(NormRopeParams p, int sms, cudaStream_t stream) {
  if (!p.n_freq) p.rot_start = 0;
  int grid = 0;
  const cudaError_t e = by_width(p, [&](auto g, auto np, auto nm) {
    constexpr int G = decltype(g)::value, NP = decltype(np)::value, NM = decltype(nm)::value;
    p.tokens_per_block = tokens_per_block(p, kBwdThreads / G, sms);
    const long long chunks = ((long long)p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
    const long long most = norm_rope_bwd_blocks(sms);
    grid = (int)(chunks < most ? chunks : most);
    size_t smem = (size_t)p.tokens_per_block * p.n_freq * 16;
    const size_t red = (size_t)(kBwdThreads / 32) * p.norm_dim * 4;
    if (red > smem) smem = red;
    return launch_pdl(p.b ? norm_rope_bwd_kernel<G, NP, NM, true> : norm_rope_bwd_kernel<G, NP, NM, false>, dim3(grid), dim3(kBwdThreads), smem, stream, p);
  });
  if (e != cudaSuccess || p.norm == DSA_NORM_NONE) return e;
  return launch_pdl(norm_rope_sum_kernel, dim3((p.norm_dim + 31) / 32, p.b ? 2 : 1), dim3(256), 0, stream, p, grid);
}

}  // namespace dsa
