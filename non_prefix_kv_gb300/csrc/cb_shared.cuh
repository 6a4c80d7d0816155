// What the kernels of the shared-prefix attention have in common.
#pragma once
#include <math.h>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"

namespace cb {

constexpr int kMaxGroups = 64;

// The call as the kernels see it.
struct Shared {
  const void* q;                 // [n_seq, n_q, H hd]
  const int32_t* last;           // [n_seq, n_q]
  void* out;
  const void *k, *v;             // the prefixes' rows
  const void *own_k, *own_v;     // [n_seq, capacity, Hkv hd]
  int64_t capacity, n_rows;
  int n_seq, n_q, H, Hkv, G, hd, n_groups;
  float scale_log2;              // log2(e) / sqrt(hd)
  int32_t row0[kMaxGroups], len[kMaxGroups], seq0[kMaxGroups + 1];
};

// the last own row that query t = s n_q + j sees: -1 none, -2 not even the prefix; a bad one counts as -2
__device__ __forceinline__ int shared_last(const Shared& p, int64_t t) {
  const int l = p.last[t];
  return l < -2 || l >= p.capacity ? -2 : l;
}

// A line of `total` steps cut into equal runs for n workers (n <= 2^12): the first step of worker w's,
// floor(total w / n), and the worker whose run holds step x.
__device__ __forceinline__ int run_start(int total, int w, int n) {
  const unsigned each = (unsigned)total / (unsigned)n, rest = (unsigned)total - each * n;
  return (int)(each * w + rest * w / n);
}
__device__ __forceinline__ int worker_of(int total, int x, int n) {
  // the largest w with floor(total w / n) <= x, that is total w < (x + 1) n
  const int64_t a = ((int64_t)x + 1) * n - 1;
  int w = (int)__fdividef((float)a, (float)total);           // off by less than one
  if ((int64_t)w * total > a) --w;
  if ((int64_t)(w + 1) * total <= a) ++w;
  return w;
}

// cb_shared.cu
size_t shared_simt_ws_bytes(const Shared& p);
cudaError_t launch_shared_simt(int dt, const Shared& p, void* ws, cudaStream_t s);
// cb_shared_tc.cu
bool shared_tc_taken(int dt, const Shared& p);
size_t shared_tc_ws_bytes(const Shared& p);
cudaError_t launch_shared_tc(const Shared& p, void* ws, cudaStream_t s);
int shared_tc_launches(const Shared& p);

}  // namespace cb
