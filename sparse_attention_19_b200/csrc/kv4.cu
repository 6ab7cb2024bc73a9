// kv4.cu -- the latent cache in 4 bits: storing rows and reading them back.
//
// A latent row has d_v value columns and a tail of d_qk - d_v (rotated) columns.  The
// value columns are held in groups of 32 as integers q in -7..7 times one bf16 step:
//   step = max|x| / 7 rounded up to 5 significant bits,   q = rne(x / step),
//   value = q * step.
// Rounding the step up keeps |x / step| <= 7 (nothing is clipped), and 5 bits of step
// times 3 bits of q fit bf16's 8, so the value is exact in bf16 and a reader may feed it
// to a bf16 matrix product unrounded.  The tail stays bf16: the rotation puts position
// into it, which 4 bits would lose.
// A group whose largest magnitude is below 2^-100 is stored as zeros; one that holds a
// NaN, an infinity or a magnitude above 2^126 has a NaN step and reads back as NaN.
//
// Row layout, chosen for the attention's loader (one thread then holds 16 columns of
// every 64-column chunk in consecutive bytes): nibble = q + 8; with chunk c = col / 64,
// part p = col / 16 % 4, word w = col / 8 % 2, the 8 columns of a word sit in the 4 bytes
// at p * (d_v / 8) + c * 8 + w * 4, column e of the word in nibble e / 2 + 4 * (e % 2).
// The step of group g = col / 32 is entry (g % 2) * (d_v / 64) + g / 2.
//
// A thread holds 16 columns, so a warp reads and writes whole rows (1152 bytes in, 416 out for
// 576 columns, or the reverse).  32768 rows, caches cold, floor 7.9 us by HBM bytes: the store takes
// 15.1 us, bound by issue slots (72 %: both lanes of a group compute its step and reciprocal; DRAM
// 31 %); the read-back 13.7 us, bound by the latency of its loads and by L1 (69 %; issue 45 %).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dsa_internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 7.888609052210118e-31f;       // 2^-100
constexpr uint32_t kHugeBits = 0x7e800000u;           // bits of 2^126

// Row and column share of a thread: LANES threads of 16 columns per row.
template <int DV>
struct Share {
  static constexpr int kLanes = DV / 16;
  static constexpr int kRows = kThreads / kLanes;     // rows per block
};

// Cache row of input row `row`, or -1 when it lies outside the cache.
__device__ __forceinline__ long long cache_row(const Kv4Params& p, int row) {
  const int b = p.div_l(row), i = row - b * p.L;
  const long long r = (long long)(p.start ? __ldg(p.start + b) : p.offset) + i;
  return r >= 0 && r < p.Lk ? (long long)b * p.Lk + r : -1;
}

template <int DV>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4Params p) {
  using S = Share<DV>;
  const int lane = threadIdx.x % S::kLanes;           // columns 16 lane .. 16 lane + 15
  const int row = (int)blockIdx.x * S::kRows + threadIdx.x / S::kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const bool here = row < p.B * p.L;
  const long long at = here ? cache_row(p, row) : -1;
  const uint4* src = reinterpret_cast<const uint4*>(p.in + (size_t)(here ? row : 0) * p.d_qk);
  uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, t = v[0];
  const int tail8 = (p.d_qk - DV) / 8;                // 16-byte vectors of the tail
  if (at >= 0) {
    v[0] = __ldg(src + 2 * lane);
    v[1] = __ldg(src + 2 * lane + 1);
    if (lane < tail8) t = __ldg(src + DV / 8 + lane);
  }
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  float2 x[8];
  uint32_t m = 0;                                     // largest magnitude as an integer: a NaN wins
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    m = max(m, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));     // the group's other 16 columns
  float step = __uint_as_float((__float_as_uint(__fdiv_rn(__uint_as_float(m), 7.f)) + 0x7ffffu) & ~0x7ffffu);
  const bool zero = __uint_as_float(m) < kTiny, bad = m > kHugeBits;
  if (zero) step = 0.f;
  if (bad) step = __uint_as_float(0x7fc00000u);
  uint32_t code[2] = {0x88888888u, 0x88888888u};
  if (!zero && !bad) {
    // The quotient as one multiplication by the rounded reciprocal and Markstein's correction
    // by the residual (exact in a fused multiply-add), which rounds it correctly: a value
    // halfway between two codes stays there.  Adding 1.5 * 2^23 + 8 then rounds it to
    // the nearest integer, ties to even, and leaves q + 8 in the sum's low bits.
    const float r = __frcp_rn(step);
    const float2 inv = make_float2(r, r), neg = make_float2(-step, -step);
    const float2 magic = make_float2(12582920.f, 12582920.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      code[k] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {                   // columns 2i and 2i + 1: nibbles i and i + 4
        const float2 v = x[4 * k + i], q0 = fmul2(v, inv);
        const float2 n = fadd2(ffma2(ffma2(q0, neg, v), inv, q0), magic);
        const uint32_t both = (__float_as_uint(n.x) & 15u) | ((__float_as_uint(n.y) & 15u) << 16);
        code[k] |= both << (4 * i);
      }
    }
  }
  if (at < 0) return;
  const int c = lane / 4, part = lane % 4;
  *reinterpret_cast<uint2*>(p.codes + (size_t)at * (DV / 2) + part * (DV / 8) + c * 8) = make_uint2(code[0], code[1]);
  if (part % 2 == 0)
    p.scales[(size_t)at * (DV / 32) + (part / 2) * (DV / 64) + c] = __float2bfloat16_rn(step);
  if (lane < tail8) reinterpret_cast<uint4*>(p.tail + (size_t)at * (p.d_qk - DV))[lane] = t;
}

// A thread has its share of two rows in flight (one: 13.5 us for 32768 rows, waiting for loads).
constexpr int kReadRows = 2;
template <int DV>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Params p) {
  using S = Share<DV>;
  const int lane = threadIdx.x % S::kLanes;
  const int row0 = (int)blockIdx.x * S::kRows * kReadRows + threadIdx.x / S::kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const int tail8 = (p.d_qk - DV) / 8, c = lane / 4, part = lane % 4, n = p.B * p.L;
  const int n_out = n + p.zero_rows;
  uint2 code[kReadRows];
  uint32_t step[kReadRows];
  uint4 t[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int row = row0 + i * S::kRows;
    const long long at = row < n ? cache_row(p, row) : -1;
    code[i] = make_uint2(0, 0);
    step[i] = 0;                                      // a step of 0: zeros
    t[i] = make_uint4(0, 0, 0, 0);
    if (at >= 0) {
      code[i] = __ldg(reinterpret_cast<const uint2*>(p.codes + (size_t)at * (DV / 2) + part * (DV / 8) + c * 8));
      step[i] = reinterpret_cast<const unsigned short*>(p.scales)[(size_t)at * (DV / 32) + (part / 2) * (DV / 64) + c];
      if (lane < tail8) t[i] = __ldg(reinterpret_cast<const uint4*>(p.tail + (size_t)at * (p.d_qk - DV)) + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int row = row0 + i * S::kRows;
    if (row >= n_out) return;
    const Kv4Step s = kv4_step(step[i]);
    uint4* dst = reinterpret_cast<uint4*>(p.out + (size_t)row * p.d_qk);
    dst[2 * lane] = unpack_codes(code[i].x, s);
    dst[2 * lane + 1] = unpack_codes(code[i].y, s);
    if (lane < tail8) dst[DV / 8 + lane] = t[i];
  }
}

unsigned blocks(const Kv4Params& p, int rows_per_block) {
  return (unsigned)(((long long)p.B * p.L + p.zero_rows + rows_per_block - 1) / rows_per_block);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Params& p, cudaStream_t stream) {
  if (p.d_v == 512)
    return launch_pdl(kv4_write_kernel<512>, dim3(blocks(p, Share<512>::kRows)), dim3(kThreads), 0, stream, p);
  return launch_pdl(kv4_write_kernel<128>, dim3(blocks(p, Share<128>::kRows)), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_kv4_read(const Kv4Params& p, cudaStream_t stream) {
  if (p.d_v == 512)
    return launch_pdl(kv4_read_kernel<512>, dim3(blocks(p, Share<512>::kRows * kReadRows)), dim3(kThreads), 0, stream, p);
  return launch_pdl(kv4_read_kernel<128>, dim3(blocks(p, Share<128>::kRows * kReadRows)), dim3(kThreads), 0, stream, p);
}

}  // namespace dsa
