// Device helpers of the 8-bit block-scaled KV cache, shared by its kernels.
#pragma once
#include <cuda_fp16.h>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"

namespace cb {

constexpr float kKv8MinScale = 1e-8f;

// The integer nearest to x / s (ties to even), s > 0, inv ~ 1/s: rint(x * inv) is within one
// of it, and the residual x - c s is exact in one fma (|r| <= s/2 and r is a multiple of the
// smaller of the two operands' last places), so comparing it with s/2 decides.
__device__ __forceinline__ float kv8_code(float x, float s, float inv) {
  float c = rintf(x * inv);
  const float r = fmaf(-c, s, x), h = 0.5f * s;
  const bool odd = ((int)c & 1) != 0;
  if (r > h || (r == h && odd))
    c += 1.0f;
  else if (r < -h || (r == -h && odd))
    c -= 1.0f;
  return fminf(fmaxf(c, -127.0f), 127.0f);
}

// The integer nearest to c0 * old / s for a code c0 (old <= s): both products of the residual
// are exact in fp64 (31 bits), and so is their difference.
__device__ __forceinline__ float kv8_recode(float c0, float old, float s, float inv) {
  float c = rintf(c0 * old * inv);
  const double r = (double)c0 * (double)old - (double)c * (double)s, h = 0.5 * (double)s;
  const bool odd = ((int)c & 1) != 0;
  if (r > h || (r == h && odd))
    c += 1.0f;
  else if (r < -h || (r == -h && odd))
    c -= 1.0f;
  return fminf(fmaxf(c, -127.0f), 127.0f);
}

// 4 codes of a word as floats: byte ^ 0x80 = c + 128 under the exponent of 2^23 (no conversion
// instruction: those run at a quarter of the rate)
__device__ __forceinline__ void kv8_unpack4(uint32_t w, float* f) {
  const uint32_t u = w ^ 0x80808080u;
  f[0] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - 8388736.0f;
  f[1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - 8388736.0f;
  f[2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - 8388736.0f;
  f[3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - 8388736.0f;
}
__device__ __forceinline__ void kv8_unpack16(const uint4 u, float* f) {
  kv8_unpack4(u.x, f);
  kv8_unpack4(u.y, f + 4);
  kv8_unpack4(u.z, f + 8);
  kv8_unpack4(u.w, f + 12);
}
__device__ __forceinline__ uint32_t kv8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // low bytes
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes of 16 values: x inv + 1.5 2^23 leaves the nearest integer in the low byte (a
// two's-complement byte, as the 24 bits above it hold the offset's); its distance tells whether
// the rounding of inv (at most 127 2^-23 in the quotient) could have chosen the other one.  Only
// then, about one value in 4000, the exact decision is taken.
__device__ __forceinline__ uint4 kv8_code16(const float* x, float s, float inv) {
  constexpr float kMagic = 12582912.0f;
  uint32_t q[16];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float t = fmaf(x[i], inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(x[i], inv, kMagic - t)));
    q[i] = __float_as_uint(t);
  }
  if (far > 0.5f - 3.1e-5f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = (uint32_t)(int)kv8_code(x[i], s, inv);
  }
  return make_uint4(kv8_pack4(q[0], q[1], q[2], q[3]), kv8_pack4(q[4], q[5], q[6], q[7]),
                    kv8_pack4(q[8], q[9], q[10], q[11]), kv8_pack4(q[12], q[13], q[14], q[15]));
}

// block-wide maximum of non-negative values (whole warps); sh holds one float per warp
__device__ __forceinline__ float kv8_block_max(float v, float* sh) {
  v = warp_max(v);
  const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) sh[w] = v;
  __syncthreads();
  float m = 0.f;
  for (int i = 0; i < nw; ++i) m = fmaxf(m, sh[i]);
  return m;
}

}  // namespace cb
