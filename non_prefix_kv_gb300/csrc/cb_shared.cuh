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
  int64_t capacity;
  int n_seq, n_q, H, Hkv, G, hd, n_groups;
  float scale_log2;              // log2(e) / sqrt(hd)
  int32_t row0[kMaxGroups], len[kMaxGroups], seq0[kMaxGroups + 1];
};

// the last own row that query t = s n_q + j sees: -1 none, -2 not even the prefix; a bad one counts as -2
__device__ __forceinline__ int shared_last(const Shared& p, int64_t t) {
  const int l = p.last[t];
  return l < -2 || l >= p.capacity ? -2 : l;
}

}  // namespace cb
