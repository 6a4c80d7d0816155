// Device helpers of the 8-bit block-scaled KV cache, shared by its kernels.
#pragma once
#include <cuda_fp16.h>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_tc.cuh"

namespace cb {

constexpr float kKv8MinScale = 1e-8f;

// The integer nearest to x / s (ties to even), s > 0, as the low byte, from q = the bits of
// c + 1.5 2^23 with c within one of it: the residual x - c s is exact in one fma (|r| <= s and
// r is a multiple of the smaller of the two operands' last places).  Beyond s/2, or at s/2 and c
// odd (the same as beyond the float before s/2), the neighbour is nearer.
__device__ __forceinline__ uint32_t kv8_code(float x, float s, uint32_t q) {
  const float r = fmaf(12582912.0f - __uint_as_float(q), s, x);
  if (fabsf(r) > __uint_as_float(__float_as_uint(0.5f * s) - (q & 1u))) q += (__float_as_int(r) >> 31) | 1;
  return q;
}

// The same for c0 * old / s of a code c0 (old <= s): both products of the residual are exact in
// fp64 (31 bits), and so is their difference.
__device__ __forceinline__ uint32_t kv8_recode(float c0, float old, float s, uint32_t q) {
  const double r = (double)c0 * (double)old + (double)(12582912.0f - __uint_as_float(q)) * (double)s, h = 0.5 * (double)s;
  if (fabs(r) > h || (fabs(r) == h && (q & 1u))) q += r > 0.0 ? 1u : ~0u;
  return q;
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the part of (a, b) that their fp16 rounding p leaves over, again as an fp16 pair
__device__ __forceinline__ uint32_t rest_h2(float a, float b, uint32_t p) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
  return pack_h2(a - f.x, b - f.y);
}

// 16 codes as 8 pairs of floats: byte ^ 0x80 = c + 128 under the exponent of 2^23 (no conversion
// instruction: those run at a quarter of the rate)
__device__ __forceinline__ void kv8_unpack16(const uint4 v, uint64_t* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t off = tc::f2_pack(-8388736.0f, -8388736.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    f[2 * i] = tc::f2_add(tc::f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)),
                                      __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441))), off);
    f[2 * i + 1] = tc::f2_add(tc::f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)),
                                          __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443))), off);
  }
}
__device__ __forceinline__ uint32_t kv8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // low bytes
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes of 16 values, whose quotients by the scale are x * inv up to 3 roundings:
// x inv + 1.5 2^23 leaves the nearest integer in the low byte (a two's-complement byte, as the
// 24 bits above it hold the offset's); its distance tells whether the roundings (at most
// 127 * 3 * 2^-24 = 2.3e-5 in the quotient) could have chosen the other one.  Only then
// exact(value, code) decides, for the 4 values of a word: one value in 16000 by chance, but
// half a block's largest value is a tie, which bf16 values hit often, and re-coded rows of one
// old block nearly always.
template <typename F>
__device__ __forceinline__ uint4 kv8_code16(const uint64_t* x, float inv, F&& exact) {
  constexpr float kMagic = 12582912.0f;
  const uint64_t inv2 = tc::f2_pack(inv, inv), magic = tc::f2_pack(kMagic, kMagic), minus = tc::f2_pack(-1.f, -1.f);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t0 = tc::f2_fma(x[2 * i], inv2, magic), t1 = tc::f2_fma(x[2 * i + 1], inv2, magic);
    const float2 d0 = tc::f2_unpack(tc::f2_fma(x[2 * i], inv2, tc::f2_fma(t0, minus, magic)));
    const float2 d1 = tc::f2_unpack(tc::f2_fma(x[2 * i + 1], inv2, tc::f2_fma(t1, minus, magic)));
    const float2 c0 = tc::f2_unpack(t0), c1 = tc::f2_unpack(t1);
    uint32_t q[4] = {__float_as_uint(c0.x), __float_as_uint(c0.y), __float_as_uint(c1.x), __float_as_uint(c1.y)};
    if (fmaxf(fmaxf(fabsf(d0.x), fabsf(d0.y)), fmaxf(fabsf(d1.x), fabsf(d1.y))) > 0.5f - 3.1e-5f) {
      const float2 v0 = tc::f2_unpack(x[2 * i]), v1 = tc::f2_unpack(x[2 * i + 1]);
      q[0] = exact(v0.x, q[0]);
      q[1] = exact(v0.y, q[1]);
      q[2] = exact(v1.x, q[2]);
      q[3] = exact(v1.y, q[3]);
    }
    w[i] = kv8_pack4(q[0], q[1], q[2], q[3]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// block-wide maximum of non-negative values as their bits (whole warps); sh holds one word per warp
__device__ __forceinline__ float kv8_block_max(uint32_t v, uint32_t* sh) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return __uint_as_float(__reduce_max_sync(0xffffffffu, lane < nw ? sh[lane] : 0u));
}

}  // namespace cb
