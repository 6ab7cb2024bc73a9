// kv4.cuh -- 8 columns of the 4-bit latent cache as bf16 (used by the cache's reader and by
// the attention over it).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

namespace dsa {

// A group's step as a pair, and what unpack_codes subtracts.
struct Kv4Step {
  __nv_bfloat162 s, off;
};
__device__ __forceinline__ Kv4Step kv4_step(uint32_t bf16_bits) {
  const uint32_t dup = bf16_bits | (bf16_bits << 16);
  Kv4Step t;
  t.s = *reinterpret_cast<const __nv_bfloat162*>(&dup);
  t.off = __hmul2(t.s, __floats2bfloat162_rn(-24.f, -24.f));
  return t;
}

// Nibble n stands for n - 8: put at bits 3-6 of bf16's 16.0 it makes 16 + n, and one fused
// multiply-add (16 + n) * s - 24 s gives (n - 8) s exactly, since s has 5 significant bits
// and |n - 8| 3 (and 24 s is exact).  A word's columns 2k and 2k + 1 are nibbles k and k + 4, so one
// shift and one logic operation place both.
__device__ __forceinline__ uint4 unpack_codes(uint32_t w, const Kv4Step& t) {
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t sh = k == 0 ? w << 3 : w >> (4 * k - 3);
    uint32_t b = (sh & 0x00780078u) | 0x41804180u;
    __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&b);
    v = __hfma2(v, t.s, t.off);
    r[k] = *reinterpret_cast<uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace dsa
