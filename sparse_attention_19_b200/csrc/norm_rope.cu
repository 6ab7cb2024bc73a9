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
// Both are bound by HBM: 2 bytes read and 1 or 2 written per element (gradient: 4 read,
// 2 written) against some 20 fp32 operations.  G lanes hold a row (16-byte vectors, N per
// lane), so a row's sums are shuffles within G lanes; every group has R rows in flight
// so that a block of 256 threads keeps 16 KB of loads outstanding.  The angles of a
// block's tokens are computed once (64-bit range reduction, so a position of 2^31 is as
// exact as a small one) into shared memory while those loads are in flight; all heads of
// a token share them.  The other half of a rotated pair is loaded again (an L1 hit)
// instead of exchanged between lanes: the pairing then works for any split of a row over
// lanes.
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
constexpr uint32_t kAmaxFloor = 0x0DA24260u;   // bits of 1e-30f: an all-zero token keeps a positive scale

struct Vec8 {
  float v[8];
};

__device__ __forceinline__ Vec8 unpack8(const uint4& u) {
  Vec8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint4 pack8(const Vec8& a) {
  return make_uint4(pack2(a.v[0], a.v[1]), pack2(a.v[2], a.v[3]), pack2(a.v[4], a.v[5]), pack2(a.v[6], a.v[7]));
}

// 8 parameters from column c (16-byte aligned in either type).
__device__ __forceinline__ Vec8 load_param8(const void* w, int is_bf16, int c) {
  if (is_bf16) return unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c)));
  Vec8 r;
  const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
  const float4 a = __ldg(p), b = __ldg(p + 1);
  r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
  r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
  return r;
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of the tokens [tok0, tok0 + ntok) for every frequency.  Entry j of a token
// sits at (j % 8) * (F / 8) + j / 8, so that lanes with neighbouring vectors read
// neighbouring words.
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int tok0, int ntok, float* cs, float* sn) {
  const int F = p.n_freq, V = F / 8;
  for (int x = threadIdx.x; x < ntok * F; x += blockDim.x) {
    const int tl = x / F, j = x - tl * F;
    const int tok = tok0 + tl;
    const int pos = p.positions ? __ldg(p.positions + tok) : p.q_offset + tok % p.L;
    const double turns = (double)pos * ((double)__ldg(p.inv_freq + j) * 0.15915494309189533577);
    const float part = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * part, &s, &c);
    const int at = tl * F + (j & 7) * V + (j >> 3);
    cs[at] = c;
    sn[at] = s;
  }
}

// Where vector `vec` of a row lies in the rotated range.
struct RotSpot {
  bool in;        // inside the rotated range
  bool second;    // half-split: the b member of the pairs
  int partner;    // half-split: vector that holds the other member
  int j8;         // first frequency / 8 (half-split), / 4 (interleaved: 4 frequencies a vector)
};
__device__ __forceinline__ RotSpot rot_spot(const NormRopeParams& p, int vec) {
  RotSpot r;
  const int v = vec - p.rot_start / 8, V = p.n_freq / 8;
  r.in = p.n_freq > 0 && v >= 0 && v < 2 * V;
  r.second = v >= V;
  r.partner = r.second ? vec - V : vec + V;
  r.j8 = p.interleaved ? v : (r.second ? v - V : v);
  return r;
}

// y = z turned by the token's angles; `sign` -1 turns back.  `o` is the other member's
// vector (half-split only).
__device__ __forceinline__ Vec8 rotate8(const NormRopeParams& p, const RotSpot& s, const Vec8& z, const Vec8& o,
                                        const float* cs, const float* sn, float sign) {
  const int V = p.n_freq / 8;
  Vec8 y;
  if (p.interleaved) {
    // vector v holds pairs 4v .. 4v+3; frequency j sits at (j % 8) * V + j / 8
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = s.j8 * 4 + e;
      const float c = cs[(j & 7) * V + (j >> 3)], t = sign * sn[(j & 7) * V + (j >> 3)];
      y.v[2 * e] = z.v[2 * e] * c - z.v[2 * e + 1] * t;
      y.v[2 * e + 1] = z.v[2 * e + 1] * c + z.v[2 * e] * t;
    }
  } else {
    const float flip = s.second ? sign : -sign;
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] = z.v[e] * cs[e * V + s.j8] + o.v[e] * (flip * sn[e * V + s.j8]);
  }
  return y;
}

// Mean and 1/std of a row held by G lanes.
template <int G, int N>
__device__ __forceinline__ void row_stats(const NormRopeParams& p, const uint4 (&raw)[N], int lane, float& mean,
                                          float& rstd) {
  mean = 0.f;
  rstd = 1.f;
  if (p.norm == DSA_NORM_NONE) return;
  const float inv_n = 1.f / (float)p.norm_dim;
  if (p.norm == DSA_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Vec8 x = unpack8(raw[n]);
      if ((n * G + lane) * 8 < p.norm_dim)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x.v[e];
    }
    mean = group_sum<G>(s) * inv_n;
  }
  float q = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Vec8 x = unpack8(raw[n]);
    if ((n * G + lane) * 8 < p.norm_dim)
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(x.v[e] - mean, x.v[e] - mean, q);
  }
  rstd = rsqrtf(group_sum<G>(q) * inv_n + p.eps);
}

// Rows of one block: tokens [tok0, tok0 + ntok), all heads, in steps of R rows per group.
template <int G, int N, int R, bool E4M3>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int kGroups = kThreads / G;
  extern __shared__ float smem[];
  float* cs = smem;
  float* sn = cs + p.tokens_per_block * p.n_freq;
  uint32_t* amax = reinterpret_cast<uint32_t*>(sn + p.tokens_per_block * p.n_freq);   // per token (e4m3)
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int tok0 = (int)blockIdx.x * p.tokens_per_block;
  const int ntok = min(p.tokens_per_block, p.n_tokens - tok0);
  const int rows = ntok * p.H;
  const int steps = (rows + kGroups * R - 1) / (kGroups * R);
  griddep_launch_dependents();
  griddep_wait();
  if (E4M3)
    for (int t = threadIdx.x; t < ntok; t += kThreads) amax[t] = kAmaxFloor;

  uint4 raw[R][N], other[R][N];
  float y[R][N][8];
  // e4m3 needs the token's maximum before its first code.  A block whose rows fit one step
  // keeps them in registers; a token of more rows is computed twice, the second time
  // from L2.
  const int passes = (E4M3 && steps > 1) ? 2 : 1;
  for (int pass = 0; pass < passes; ++pass) {
    for (int st = 0; st < steps; ++st) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = st * kGroups * R + i * kGroups + group;
        const int tl = row < rows ? row / p.H : 0, h = row < rows ? row - tl * p.H : 0;
        const int tok = tok0 + tl, b = tok / p.L, l = tok - b * p.L;
        const __nv_bfloat16* src = p.x + b * p.stride_b + l * p.stride_l + h * p.stride_h;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int vec = n * G + lane;
          raw[i][n] = other[i][n] = make_uint4(0, 0, 0, 0);
          if (row < rows && vec * 8 < p.D) {
            raw[i][n] = __ldg(reinterpret_cast<const uint4*>(src) + vec);
            const RotSpot s = rot_spot(p, vec);
            if (s.in && !p.interleaved) other[i][n] = __ldg(reinterpret_cast<const uint4*>(src) + s.partner);
          }
        }
      }
      if (pass == 0 && st == 0) {
        fill_angles(p, tok0, ntok, cs, sn);
        __syncthreads();
      }
      float mean[R], rstd[R];
#pragma unroll
      for (int i = 0; i < R; ++i) row_stats<G, N>(p, raw[i], lane, mean[i], rstd[i]);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int vec = n * G + lane;
        const RotSpot s = rot_spot(p, vec);
        const bool normed = p.norm != DSA_NORM_NONE && vec * 8 < p.norm_dim;
        const bool onormed = p.norm != DSA_NORM_NONE && s.in && s.partner * 8 < p.norm_dim;
        Vec8 w{}, bias{}, ow{}, obias{};
        if (normed) {
          w = load_param8(p.w, p.w_bf16, vec * 8);
          if (p.b) bias = load_param8(p.b, p.w_bf16, vec * 8);
        }
        if (onormed && !p.interleaved) {
          ow = load_param8(p.w, p.w_bf16, s.partner * 8);
          if (p.b) obias = load_param8(p.b, p.w_bf16, s.partner * 8);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int row = st * kGroups * R + i * kGroups + group;
          const int tl = row < rows ? row / p.H : 0;
          Vec8 z = unpack8(raw[i][n]), o = unpack8(other[i][n]);
          if (normed)
#pragma unroll
            for (int e = 0; e < 8; ++e) z.v[e] = fmaf((z.v[e] - mean[i]) * rstd[i], w.v[e], bias.v[e]);
          if (onormed)
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] = fmaf((o.v[e] - mean[i]) * rstd[i], ow.v[e], obias.v[e]);
          if (s.in) z = rotate8(p, s, z, o, cs + tl * p.n_freq, sn + tl * p.n_freq, 1.f);
          if (!E4M3) {
            if (row < rows && vec * 8 < p.D)
              *reinterpret_cast<uint4*>(p.out + ((size_t)tok0 * p.H + row) * p.D + vec * 8) = pack8(z);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][n][e] = z.v[e];
          }
        }
      }
      if (E4M3 && pass == 0) {
        // Maximum of |y| as integers: it does not depend on the order, and a NaN wins.
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int row = st * kGroups * R + i * kGroups + group;
          uint32_t m = 0;
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(y[i][n][e]) & 0x7fffffffu);
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (lane == 0 && row < rows) atomicMax(&amax[row / p.H], m);
        }
        if (st == steps - 1) {
          __syncthreads();
          for (int t = threadIdx.x; t < ntok; t += kThreads) p.scale[tok0 + t] = __uint_as_float(amax[t]) / 448.f;
        }
      }
      if (E4M3 && pass == passes - 1) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int row = st * kGroups * R + i * kGroups + group;
          if (row >= rows) continue;
          // y / scale as y * (1 / scale): at most one fp32 step from the quotient.
          const float inv = 1.f / (__uint_as_float(amax[row / p.H]) / 448.f);
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const int vec = n * G + lane;
            if (vec * 8 >= p.D) continue;
            uint32_t code[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              code[e] = __nv_cvt_float2_to_fp8x2(make_float2(y[i][n][2 * e] * inv, y[i][n][2 * e + 1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<uint2*>(p.codes + ((size_t)tok0 * p.H + row) * p.D + vec * 8) =
                make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
          }
        }
      }
    }
  }
}

// Gradient.  Persistent blocks: each walks its chunks of tokens, keeps the sums for dw
// and db of its columns in registers, and leaves one partial row per block; a second
// kernel adds the partial rows in block order, so the result does not depend on timing.
template <int G, int N, int R>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeParams p) {
  constexpr int kGroups = kThreads / G;
  extern __shared__ float smem[];
  const int table = p.tokens_per_block * p.n_freq;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  griddep_launch_dependents();
  griddep_wait();
  float dw[N][8], db[N][8];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[n][e] = db[n][e] = 0.f;

  const int n_chunks = (int)(((long long)p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block);
  int buf = 0;
  for (int ch = blockIdx.x; ch < n_chunks; ch += gridDim.x, buf ^= 1) {
    const int tok0 = ch * p.tokens_per_block;
    const int ntok = min(p.tokens_per_block, p.n_tokens - tok0);
    const int rows = ntok * p.H;
    const int steps = (rows + kGroups * R - 1) / (kGroups * R);
    float* cs = smem + buf * 2 * table;         // two tables: the next chunk's may be filled
    float* sn = cs + table;                     // while slower warps still read this one
    for (int st = 0; st < steps; ++st) {
      uint4 raw[R][N], graw[R][N], other[R][N];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = st * kGroups * R + i * kGroups + group;
        const int tl = row < rows ? row / p.H : 0, h = row < rows ? row - tl * p.H : 0;
        const int tok = tok0 + tl, b = tok / p.L, l = tok - b * p.L;
        const __nv_bfloat16* src = p.x + b * p.stride_b + l * p.stride_l + h * p.stride_h;
        const __nv_bfloat16* gsrc = p.dy + ((size_t)tok0 * p.H + row) * p.D;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int vec = n * G + lane;
          raw[i][n] = graw[i][n] = other[i][n] = make_uint4(0, 0, 0, 0);
          if (row < rows && vec * 8 < p.D) {
            if (vec * 8 < p.norm_dim) raw[i][n] = __ldg(reinterpret_cast<const uint4*>(src) + vec);
            graw[i][n] = __ldg(reinterpret_cast<const uint4*>(gsrc) + vec);
            const RotSpot s = rot_spot(p, vec);
            if (s.in && !p.interleaved) other[i][n] = __ldg(reinterpret_cast<const uint4*>(gsrc) + s.partner);
          }
        }
      }
      if (st == 0) {
        fill_angles(p, tok0, ntok, cs, sn);
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = st * kGroups * R + i * kGroups + group;
        const int tl = row < rows ? row / p.H : 0;
        float mean, rstd;
        row_stats<G, N>(p, raw[i], lane, mean, rstd);
        float g[N][8], s1 = 0.f, s2 = 0.f;      // g = dz (behind norm_dim) or dz w; sums of g and g xhat
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int vec = n * G + lane;
          const RotSpot s = rot_spot(p, vec);
          Vec8 dz = unpack8(graw[i][n]);
          if (s.in) dz = rotate8(p, s, dz, unpack8(other[i][n]), cs + tl * p.n_freq, sn + tl * p.n_freq, -1.f);
          const bool normed = p.norm != DSA_NORM_NONE && vec * 8 < p.norm_dim;
          if (normed) {
            const Vec8 x = unpack8(raw[i][n]), w = load_param8(p.w, p.w_bf16, vec * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float xh = (x.v[e] - mean) * rstd;
              // a row past the end has dz = 0, so it adds nothing
              dw[n][e] = fmaf(dz.v[e], xh, dw[n][e]);
              db[n][e] += dz.v[e];
              g[n][e] = dz.v[e] * w.v[e];
              s1 += g[n][e];
              s2 = fmaf(g[n][e], xh, s2);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[n][e] = dz.v[e];
          }
        }
        if (p.norm != DSA_NORM_NONE) {
          const float inv_n = 1.f / (float)p.norm_dim;
          s2 = group_sum<G>(s2) * inv_n;
          s1 = p.norm == DSA_NORM_LAYER ? group_sum<G>(s1) * inv_n : 0.f;
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int vec = n * G + lane;
          if (row >= rows || vec * 8 >= p.D) continue;
          Vec8 d;
          const bool normed = p.norm != DSA_NORM_NONE && vec * 8 < p.norm_dim;
          const Vec8 x = unpack8(raw[i][n]);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            d.v[e] = normed ? rstd * (g[n][e] - s1 - (x.v[e] - mean) * rstd * s2) : g[n][e];
          *reinterpret_cast<uint4*>(p.dx + ((size_t)tok0 * p.H + row) * p.D + vec * 8) = pack8(d);
        }
      }
    }
  }
  if (p.norm == DSA_NORM_NONE) return;
  // Sum the groups of the block, column by column, in group order.
  float* red = smem;                            // [kGroups][norm_dim]
  for (int what = 0; what < (p.b ? 2 : 1); ++what) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * G + lane) * 8;
      if (c < p.norm_dim)
#pragma unroll
        for (int e = 0; e < 8; ++e) red[group * p.norm_dim + c + e] = what ? db[n][e] : dw[n][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.norm_dim; c += kThreads) {
      float s = 0.f;
      for (int gi = 0; gi < kGroups; ++gi) s += red[gi * p.norm_dim + c];
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
  if (c < p.norm_dim)
    for (int i = warp; i < n_part; i += 8) s += p.part[((size_t)what * n_part + i) * p.norm_dim + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.norm_dim) {
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    (what ? p.db : p.dw)[c] = s;
  }
}

// Lanes per row, vectors per lane and rows per group for a head of D columns.
template <typename F>
cudaError_t by_width(int D, F&& f) {
  const int nv = D / 8;
  if (nv <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  if (nv <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  if (nv <= 24) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 3>{}, std::integral_constant<int, 1>{});
  if (nv <= 32) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  if (nv <= 64) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
  if (nv <= 96) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 3>{}, std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
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
  return by_width(p.D, [&](auto g, auto n, auto r) {
    constexpr int G = decltype(g)::value, N = decltype(n)::value, R = decltype(r)::value;
    p.tokens_per_block = tokens_per_block(p, kThreads / G * R, sms);
    const long long grid = ((long long)p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
    const size_t smem = (size_t)p.tokens_per_block * (p.n_freq * 8 + 4);
    return launch_pdl(p.codes ? norm_rope_kernel<G, N, R, true> : norm_rope_kernel<G, N, R, false>,
                      dim3((unsigned)grid), dim3(kThreads), smem, stream, p);
  });
}

int norm_rope_bwd_blocks(int sms) { return sms * kNormRopeBwdBlocksPerSm; }

cudaError_t launch_norm_rope_bwd(NormRopeParams p, int sms, cudaStream_t stream) {
  int grid = 0;
  const cudaError_t e = by_width(p.D, [&](auto g, auto n, auto r) {
    constexpr int G = decltype(g)::value, N = decltype(n)::value, R = decltype(r)::value;
    constexpr int RB = R > 2 ? 2 : R;           // three loads a row: half the rows in flight
    p.tokens_per_block = tokens_per_block(p, kThreads / G * RB, sms);
    const long long chunks = ((long long)p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
    const long long most = norm_rope_bwd_blocks(sms);
    grid = (int)(chunks < most ? chunks : most);
    size_t smem = (size_t)p.tokens_per_block * p.n_freq * 16;
    const size_t red = (size_t)(kThreads / G) * p.norm_dim * 4;
    if (red > smem) smem = red;
    return launch_pdl(norm_rope_bwd_kernel<G, N, RB>, dim3(grid), dim3(kThreads), smem, stream, p);
  });
  if (e != cudaSuccess || p.norm == DSA_NORM_NONE) return e;
  return launch_pdl(norm_rope_sum_kernel, dim3((p.norm_dim + 31) / 32, p.b ? 2 : 1), dim3(256), 0, stream, p, grid);
}

}  // namespace dsa
