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

// 16 codes <-> 16 floats
__device__ __forceinline__ void kv8_unpack16(const uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) f[4 * i + b] = (float)(int8_t)(w[i] >> (8 * b));
}
__device__ __forceinline__ uint4 kv8_pack16(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) v |= ((uint32_t)(int)f[4 * i + b] & 255u) << (8 * b);
    w[i] = v;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
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
