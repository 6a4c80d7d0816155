// The rules on a batch's logits before the next token (penalties for repeated ids, biases, a
// grammar's mask) and that token, in one pass over the logits.
//
// HBM-bound: a row reads and writes vocab elements and reads its mask bits and history once
// per CTA.  One cluster of CTAs per row, each owning a slice of the vocabulary: it counts the
// row's history ids that fall into its slice in shared memory (integers, so the order of the
// atomics does not matter), adds up the biases there in list order, then streams the slice
// through the rules.  The slices' best (value, id) keys meet in the cluster's shared memory,
// so there is no second launch and no workspace.  Sixteen small CTAs per row (32 KB of shared
// memory, 256 threads) let 64 rows of 64000 ids run as one wave.
#include <math.h>

#include <mutex>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_logits;

uint32_t take_error_logits() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_logits, sizeof(v)) != cudaSuccess) return ERRBIT_INDEX;
  cudaMemcpyToSymbol(g_err_logits, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;                 // ids a CTA holds counts and biases of at once
constexpr int kMaxBias = 4096;
constexpr int kMaxCluster = 16;
constexpr uint32_t kSeen = 0x80000000u;      // in the prompt (the low bits: times in the answer)
constexpr uint32_t kNoBias = 0xffffffffu;    // bias word of an id without one (no sum is stored as this NaN)
constexpr uint32_t kShared = 0x80000000u;    // on the way: more than one entry has this id

// larger value first, then the lower id; 0 only for "nothing"
__device__ __forceinline__ unsigned long long token_key(float v, int id) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 counts as +0
  const uint32_t o = (u >> 31) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)o << 32) | (uint32_t)~id;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_logits(const T* logits, T* out, int32_t* __restrict__ token, int vocab,
                                                     int slice, bool vec, const cb_logit_rules r) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = 16 / sizeof(T);          // elements of a 16-byte access
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* cnt = smem;                      // [kChunk]
  uint32_t* bias = smem + kChunk;            // [kChunk] bits of the sum, or kNoBias
  __shared__ unsigned long long s_best[kThreads / 32];
  __shared__ unsigned long long s_key;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x, row = blockIdx.y;
  const bool report = rank == 0 && tid == 0;
  const T* x = logits + (int64_t)row * vocab;
  T* y = out ? out + (int64_t)row * vocab : nullptr;
  const bool hist = r.history != nullptr, biased = r.n_bias > 0;

  int len = 0, plen = 0;
  if (hist) {
    const int64_t l = r.history_len[row], p = r.prompt_len ? r.prompt_len[row] : 0;
    len = (int)(l < 0 ? 0 : (l > r.history_ld ? r.history_ld : l));
    plen = (int)(p < 0 ? 0 : (p > len ? len : p));
    if (report && (len != l || plen != p)) atomicOr(&g_err_logits, ERRBIT_INDEX);
  }
  float rep = r.repetition ? r.repetition[row] : 1.0f;
  if (!(rep > 0.0f) || isinf(rep)) {
    if (report) atomicOr(&g_err_logits, ERRBIT_NONFINITE);
    rep = 1.0f;
  }
  const float pres = r.presence ? r.presence[row] : 0.0f, freq = r.frequency ? r.frequency[row] : 0.0f;
  const uint32_t* mask = r.mask ? r.mask + (int64_t)row * r.mask_ld : nullptr;
  const int s0 = rank * slice, s1 = min(vocab, s0 + slice);
  float best_v = -INFINITY;
  int best_i = -1;
  bool bad_id = false, bad_x = false;

  for (int c0 = s0; c0 < s1; c0 += kChunk) {
    const int n = min(kChunk, s1 - c0);
    if (hist || biased) {
      for (int i = tid; i < n; i += kThreads) {
        if (hist) cnt[i] = 0;
        if (biased) bias[i] = kNoBias;
      }
      __syncthreads();
    }
    if (hist) {
      const int32_t* ids = r.history + (int64_t)row * r.history_ld;
#pragma unroll 4
      for (int i = tid; i < len; i += kThreads) {
        const int id = ids[i], k = id - c0;
        if (id < 0 || id >= vocab)
          bad_id = true;
        else if (k >= 0 && k < n) {
          if (i >= plen)
            atomicAdd(&cnt[k], 1u);
          else
            atomicOr(&cnt[k], kSeen);
        }
      }
    }
    if (biased) {
      // The first entry of an id owns its word and adds the id's entries in list order: every
      // entry puts its number in with a minimum, one that finds another there marks the word, and
      // only the owner of a marked word looks through the rest of the list.
      const int32_t* bid = r.bias_id + (int64_t)row * r.n_bias;
      const float* bv = r.bias + (int64_t)row * r.n_bias;
      auto place = [&](int i) -> int {     // an entry's word in this chunk, or -1
        const int id = bid[i];
        if (id < -1 || id >= vocab) bad_id = true;
        return id >= c0 && id - c0 < n ? id - c0 : -1;
      };
      for (int i = tid; i < r.n_bias; i += kThreads) {
        const int k = place(i);
        if (k >= 0) atomicMin(&bias[k], (uint32_t)i);
      }
      __syncthreads();
      static_assert(kMaxBias / kThreads <= 32, "a thread's entries exceed a word");
      uint32_t owned = 0;                  // bit j: this thread's j-th entry owns its word
      for (int i = tid, j = 0; i < r.n_bias; i += kThreads, ++j) {
        const int k = place(i);
        if (k < 0) continue;
        if ((bias[k] & ~kShared) == (uint32_t)i)
          owned |= 1u << j;
        else
          atomicOr(&bias[k], kShared);
      }
      __syncthreads();
      for (; owned; owned &= owned - 1) {
        const int i = tid + (__ffs(owned) - 1) * kThreads, id = bid[i];
        float sum = bv[i];
        if (bias[id - c0] & kShared) {
#pragma unroll 4
          for (int k = i + 1; k < r.n_bias; ++k)
            if (bid[k] == id) sum += bv[k];
        }
        bias[id - c0] = sum != sum ? 0x7fffffffu : __float_as_uint(sum);
      }
    }
    if (hist || biased) __syncthreads();

    // the penalties of an id with count word c, then its bias word
    auto touch = [&](float v, uint32_t c, uint32_t w) -> float {
      if (hist && c) {                     // in the prompt or in the answer
        v = v > 0.f ? v / rep : v * rep;
        const uint32_t k = c & ~kSeen;
        if (k) v -= freq * (float)k + pres;
      }
      if (biased && w != kNoBias) v += __uint_as_float(w);
      return v;
    };
    // v as it is returned; ids come in ascending order, so the first of equals stays
    auto take = [&](float v, int id) {
      bad_x |= v != v;
      if (v > best_v) {
        best_v = v;
        best_i = id;
      }
    };
    if (vec) {
      for (int i = tid * E; i < n; i += kThreads * E) {
        T e[E];
        uint32_t c[E], w[E];
        *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(x + c0 + i);
        const uint32_t open = mask ? mask[(c0 + i) >> 5] >> ((c0 + i) & 31) : 0xffffffffu;
        uint32_t any = 0;
#pragma unroll
        for (int q = 0; q < E; q += 4) {
          if (hist) {
            const uint4 u = *reinterpret_cast<const uint4*>(cnt + i + q);
            c[q] = u.x; c[q + 1] = u.y; c[q + 2] = u.z; c[q + 3] = u.w;
            any |= u.x | u.y | u.z | u.w;
          }
          if (biased) {
            const uint4 u = *reinterpret_cast<const uint4*>(bias + i + q);
            w[q] = u.x; w[q + 1] = u.y; w[q + 2] = u.z; w[q + 3] = u.w;
            any |= ~(u.x & u.y & u.z & u.w);
          }
        }
        float f[E];
#pragma unroll
        for (int q = 0; q < E; ++q) f[q] = to_f(e[q]);
        if (any) {
#pragma unroll
          for (int q = 0; q < E; ++q) f[q] = touch(f[q], hist ? c[q] : 0u, biased ? w[q] : kNoBias);
        }
#pragma unroll
        for (int q = 0; q < E; ++q) {
          e[q] = from_f<T>((open >> q) & 1 ? f[q] : -INFINITY);
          take(to_f(e[q]), c0 + i + q);
        }
        if (y) *reinterpret_cast<uint4*>(y + c0 + i) = *reinterpret_cast<const uint4*>(e);
      }
    } else {
      for (int i = tid; i < n; i += kThreads) {
        const bool open = mask ? (mask[(c0 + i) >> 5] >> ((c0 + i) & 31)) & 1 : true;
        const float f = touch(to_f(x[c0 + i]), hist ? cnt[i] : 0u, biased ? bias[i] : kNoBias);
        const T v = from_f<T>(open ? f : -INFINITY);
        take(to_f(v), c0 + i);
        if (y) y[c0 + i] = v;
      }
    }
    __syncthreads();                       // the counts are used up before the next chunk's
  }
  if (bad_id) atomicOr(&g_err_logits, ERRBIT_INDEX);
  if (bad_x) atomicOr(&g_err_logits, ERRBIT_NONFINITE);
  if (!token) return;                      // uniform over the cluster
  unsigned long long best = best_i >= 0 ? token_key(best_v, best_i) : 0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, o);
    best = k > best ? k : best;
  }
  if (lane == 0) s_best[warp] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) best = s_best[w] > best ? s_best[w] : best;
    s_key = best;
  }
  tc::cluster_sync();
  if (rank == 0 && tid == 0) {
    for (int c = 1; c < (int)gridDim.x; ++c) {
      unsigned long long k;
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(tc::mapa_shared(tc::smem_u32(&s_key), c)));
      best = k > best ? k : best;
    }
    token[row] = best ? (int32_t)~(uint32_t)best : -1;     // nothing: no value above -inf
  }
  tc::cluster_sync();                      // the key was read before its CTA ends
}

std::mutex g_logits_mu;
uint32_t g_logits_attr[64];

template <typename T>
cudaError_t launch_t(const void* logits, int n_rows, int vocab, const cb_logit_rules& r, void* out, int32_t* token,
                     cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr uint32_t bit = sizeof(T) == 4 ? 1u : 2u;
  constexpr int smem = kChunk * 8;
  {
    std::lock_guard<std::mutex> g(g_logits_mu);
    if (dev < 0 || dev >= 64 || !(g_logits_attr[dev] & bit)) {
      e = cudaFuncSetAttribute(k_logits<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k_logits<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) g_logits_attr[dev] |= bit;
    }
  }
  int nc = kMaxCluster;
  while (nc > 1 && (int64_t)nc * 512 > vocab) nc /= 2;
  const int slice = ((vocab + nc - 1) / nc + 63) & ~63;
  const uintptr_t al = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out);
  const bool vec = (int64_t)vocab * sizeof(T) % 16 == 0 && al % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, n_rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = r.history || r.n_bias > 0 ? smem : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_logits<T>, static_cast<const T*>(logits), static_cast<T*>(out), token, vocab, slice,
                            vec, r);
}

}  // namespace

void reset_logits_caches() {
  std::lock_guard<std::mutex> g(g_logits_mu);
  for (int i = 0; i < 64; ++i) g_logits_attr[i] = 0;
}

cudaError_t launch_logits(int dt, const void* logits, int n_rows, int vocab, const cb_logit_rules& r, void* out,
                          int32_t* token, cudaStream_t s) {
  if (dt == DT_BF16) return launch_t<bf16>(logits, n_rows, vocab, r, out, token, s);
  return launch_t<float>(logits, n_rows, vocab, r, out, token, s);
}

}  // namespace cb
