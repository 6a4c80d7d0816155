// The rules on a batch's logits before the next token (penalties for repeated ids, biases, a
// grammar's mask) and that token, in one pass over the logits.
//
// HBM-bound: a row reads and writes vocab elements, its mask bits, and its history once per
// CTA.  One cluster of eight CTAs per row, each owning a slice of the vocabulary.  A CTA keeps
// one word per id of its slice in shared memory: how often the id is in the answer, whether it
// is in the prompt, and which entry of the bias list owns it.  The history is counted into the
// words (integers, so the order of the atomics does not matter), every bias entry's owner adds
// up the entries of its id in list order, then the slice streams through the rules.  The
// slices' best (value, id) keys are pushed into the first CTA's shared memory: no second
// launch, no workspace.  Everything that does not depend on the launch before (the cluster's
// meeting, the clearing of the words) comes before the wait for it.
//
// Measured, 64 rows of 64000 bf16 ids, a history of 2048, 300 biases, a mask: 15.4 us (17 MB; all
// 512 CTAs in one wave, bound by the chain history -> owners -> stream -> keys), one row of 32000
// fp32 ids with a history of 4352 7.5 us.  With a word for the count and one for the bias, sixteen
// CTAs of 256 threads per row and the keys read back through two cluster barriers, 31.7 us (two
// waves; 5.3 us of it the stream itself, 5.5 the keys).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_logits;
static std::atomic<bool> g_used_logits{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_logits() { return g_used_logits ? take_word(g_err_logits) : 0u; }

namespace {

constexpr int kThreads = 512;
constexpr int kChunk = 8192;                 // ids a CTA holds words of at once
constexpr int kMaxBias = 4096;
constexpr int kMaxCluster = 8;
// an id's word: times in the answer | 1 + how far its first bias entry is from the list's end | in the prompt
constexpr uint32_t kCount = (1u << 18) - 1, kOwner = 0x1fffu << 18, kPrompt = 1u << 31;
static_assert(kMaxBias < (1 << 13), "an entry's number exceeds its field");

// larger value first, then the lower id; 0 only for "nothing"
__device__ __forceinline__ unsigned long long token_key(float v, int id) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 counts as +0
  const uint32_t o = (u >> 31) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)o << 32) | (uint32_t)~id;
}

// acquires what the other CTAs of the cluster wrote before they arrived
__device__ __forceinline__ bool wait_cluster(uint64_t* bar) {
  for (uint32_t i = 0; i < tc::kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar))
        : "memory");
    if (ok) return true;
  }
  return false;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_logits(const T* logits, T* out, int32_t* __restrict__ token, int vocab,
                                                     int slice, bool vec, bool hvec, const cb_logit_rules r) {
  constexpr int E = 4;                       // elements a thread takes at once (more would cost a CTA per SM in registers)
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* word = smem;                     // [min(slice, kChunk)]
  float* sums = reinterpret_cast<float*>(smem + (slice < kChunk ? slice : kChunk));   // [n_bias] an owner's sum
  __shared__ uint32_t s_shared[kMaxBias / 32];     // bit i: entry i owns an id that is listed again
  __shared__ unsigned long long s_best[kThreads / 32];
  __shared__ unsigned long long s_key[kMaxCluster];
  __shared__ uint64_t s_bar;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x, row = blockIdx.y;
  const bool report = rank == 0 && tid == 0;
  const bool hist = r.history != nullptr, biased = r.n_bias > 0;
  const int s0 = rank * slice, s1 = min(vocab, s0 + slice);
  auto clear = [&](int n) {
    if (hist || biased)
      for (int i = tid * 4; i < n; i += kThreads * 4) *reinterpret_cast<uint4*>(word + i) = make_uint4(0, 0, 0, 0);
    if (biased)
      for (int i = tid; i < kMaxBias / 32; i += kThreads) s_shared[i] = 0;
  };
  if (token) {
    if (tid == 0) {
      tc::mbar_init(&s_bar, gridDim.x);
      tc::fence_mbar_init();
    }
    tc::cluster_sync();
  }
  clear(min(kChunk, (s1 - s0 + 3) & ~3));
  pdl_wait();
  pdl_trigger();

  const T* x = logits + (int64_t)row * vocab;
  T* y = out ? out + (int64_t)row * vocab : nullptr;
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
  float best_v = -INFINITY;
  int best_i = -1;
  bool bad_id = false, bad_x = false;

  for (int c0 = s0; c0 < s1; c0 += kChunk) {
    const int n = min(kChunk, s1 - c0);
    if (c0 > s0) clear((n + 3) & ~3);
    if (hist || biased) __syncthreads();
    if (hist) {
      const int32_t* ids = r.history + (int64_t)row * r.history_ld;
      auto count = [&](int i, int id) {
        const int k = id - c0;
        if (id < 0 || id >= vocab)
          bad_id = true;
        else if (k >= 0 && k < n) {
          if (i >= plen)
            atomicAdd(&word[k], 1u);
          else
            atomicOr(&word[k], kPrompt);
        }
      };
      int i = tid * 4;
      if (hvec) {
#pragma unroll 2
        for (; i + 3 < len; i += kThreads * 4) {
          const int4 v = *reinterpret_cast<const int4*>(ids + i);
          count(i, v.x);
          count(i + 1, v.y);
          count(i + 2, v.z);
          count(i + 3, v.w);
        }
        for (int k = i; k < min(len, i + 4); ++k) count(k, ids[k]);
      } else {
#pragma unroll 4
        for (int k = tid; k < len; k += kThreads) count(k, ids[k]);
      }
    }
    if (biased) {
      // The first entry of an id owns it and adds the id's entries in list order: every entry
      // puts its distance from the list's end in with a maximum (the word's other fields do not
      // change meanwhile), one that finds another there marks the owner, and only a marked owner
      // (its warp) looks through the rest of the list.
      const int32_t* bid = r.bias_id + (int64_t)row * r.n_bias;
      const float* bv = r.bias + (int64_t)row * r.n_bias;
      auto place = [&](int i) -> int {     // an entry's word in this chunk, or -1
        const int id = bid[i];
        if (id < -1 || id >= vocab) bad_id = true;
        return id >= c0 && id - c0 < n ? id - c0 : -1;
      };
      __syncthreads();
      for (int i = tid; i < r.n_bias; i += kThreads) {
        const int k = place(i);
        if (k >= 0) atomicMax(&word[k], (word[k] & ~kOwner) | ((uint32_t)(r.n_bias - i) << 18));
      }
      __syncthreads();
      for (int i = tid; i < r.n_bias; i += kThreads) {
        const int k = place(i);
        if (k < 0) continue;
        const int owner = r.n_bias - (int)((word[k] & kOwner) >> 18);
        if (owner != i) atomicOr(&s_shared[owner >> 5], 1u << (owner & 31));
      }
      __syncthreads();
      for (int i0 = warp * 32; i0 < r.n_bias; i0 += kThreads) {
        const int i = i0 + lane, k = i < r.n_bias ? place(i) : -1;
        const bool own = k >= 0 && r.n_bias - (int)((word[k] & kOwner) >> 18) == i;
        float sum = own ? bv[i] : 0.f;
        // a listed-again id: its owner's warp walks the rest of the list, 32 entries at a time
        unsigned again = __ballot_sync(0xffffffffu, own && ((s_shared[i >> 5] >> (i & 31)) & 1));
        for (; again; again &= again - 1) {
          const int who = __ffs(again) - 1, id = c0 + __shfl_sync(0xffffffffu, k, who), from = i0 + who;
          for (int j0 = i0; j0 < r.n_bias; j0 += 32) {
            const int j = j0 + lane;
            const bool hit = j > from && j < r.n_bias && bid[j] == id;
            const float v = hit ? bv[j] : 0.f;
            for (unsigned m = __ballot_sync(0xffffffffu, hit); m; m &= m - 1) {
              const float w = __shfl_sync(0xffffffffu, v, __ffs(m) - 1);
              if (lane == who) sum += w;
            }
          }
        }
        if (own) sums[i] = sum;
      }
    }
    if (hist || biased) __syncthreads();

    // the rules of an id with a word that is not 0, every operation rounded (none joined to a
    // multiply-add: the token goes by these values, and a last bit decides between near ones)
    auto touch = [&](float v, uint32_t w) -> float {
      if (w & (kPrompt | kCount)) {
        v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
        if (w & kCount) v = __fsub_rn(v, __fadd_rn(__fmul_rn(freq, (float)(w & kCount)), pres));
      }
      if (w & kOwner) v = __fadd_rn(v, sums[r.n_bias - (int)((w & kOwner) >> 18)]);
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
        float f[E];
        ld4(x + c0 + i, f);
        const uint32_t open = mask ? mask[(c0 + i) >> 5] >> ((c0 + i) & 31) : 0xffffffffu;
        if (hist || biased) {
          const uint4 w = *reinterpret_cast<const uint4*>(word + i);
          if (w.x | w.y | w.z | w.w) {
            if (w.x) f[0] = touch(f[0], w.x);
            if (w.y) f[1] = touch(f[1], w.y);
            if (w.z) f[2] = touch(f[2], w.z);
            if (w.w) f[3] = touch(f[3], w.w);
          }
        }
#pragma unroll
        for (int q = 0; q < E; ++q) {
          f[q] = to_f(from_f<T>((open >> q) & 1 ? f[q] : -INFINITY));
          take(f[q], c0 + i + q);
        }
        if (y) st4(y + c0 + i, f);
      }
    } else {
      for (int i = tid; i < n; i += kThreads) {
        const bool open = mask ? (mask[(c0 + i) >> 5] >> ((c0 + i) & 31)) & 1 : true;
        const uint32_t w = hist || biased ? word[i] : 0u;
        float f = to_f(x[c0 + i]);
        if (w) f = touch(f, w);
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
  }
  // every CTA pushes its key into the first one's memory, which waits for all of them
  if (tid == 0) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::mapa_shared(tc::smem_u32(&s_key[rank]), 0)), "l"(best)
                 : "memory");
    tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&s_bar), 0));
    if (rank == 0) {
      if (!wait_cluster(&s_bar)) atomicOr(&g_err_logits, ERRBIT_TIMEOUT);
      for (int c = 0; c < (int)gridDim.x; ++c) best = s_key[c] > best ? s_key[c] : best;
      token[row] = best ? (int32_t)~(uint32_t)best : -1;     // nothing: no value above -inf
    }
  }
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
  constexpr int most = (kChunk + kMaxBias) * 4;
  {
    std::lock_guard<std::mutex> g(g_logits_mu);
    if (dev < 0 || dev >= 64 || !(g_logits_attr[dev] & bit)) {
      e = cudaFuncSetAttribute(k_logits<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) g_logits_attr[dev] |= bit;
    }
  }
  int nc = kMaxCluster;
  while (nc > 1 && (int64_t)nc * 512 > vocab) nc /= 2;
  const int slice = ((vocab + nc - 1) / nc + 63) & ~63;
  const uintptr_t al = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out);
  const bool vec = vocab % 4 == 0 && al % 16 == 0;         // every row starts where four elements may be moved at once
  const bool hvec = r.history_ld % 4 == 0 && reinterpret_cast<uintptr_t>(r.history) % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, n_rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = r.history || r.n_bias > 0 ? (size_t)(std::min(slice, kChunk) + r.n_bias) * 4 : 0;
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
                            vec, hvec, r);
}

}  // namespace

void reset_logits_caches() {
  std::lock_guard<std::mutex> g(g_logits_mu);
  for (int i = 0; i < 64; ++i) g_logits_attr[i] = 0;
}

cudaError_t launch_logits(int dt, const void* logits, int n_rows, int vocab, const cb_logit_rules& r, void* out,
                          int32_t* token, cudaStream_t s) {
  g_used_logits = true;
  if (dt == DT_BF16) return launch_t<bf16>(logits, n_rows, vocab, r, out, token, s);
  return launch_t<float>(logits, n_rows, vocab, r, out, token, s);
}

}  // namespace cb
