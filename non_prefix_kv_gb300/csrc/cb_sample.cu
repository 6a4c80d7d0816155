// The next token of each row from given random numbers: temperature, the k largest, the fewest that hold
// a share p, a least share of the largest, then the draw, in one launch and without a sort.
//
//   w_i = exp((l_i - max) / T);  order: falling logit, then rising id
//   kept = the first k of the order; of them the fewest whose weight reaches p of theirs; of them w_i >= min_p
//   token = the first kept id (ascending) whose running weight exceeds u times the kept weight
//
// Every decision compares sums of weights, and it should be the one that 64-bit arithmetic takes: with
// fp32 weights a draw over 64000 near-equal ids would fall on another id in one row of fifty.  So a weight
// is an integer, 2^42 w: 2^x by a table of 32 steps and the first terms of the series on the rest (Tang's table-driven
// method, ACM TOMS 15, 1989), with 31 bits behind the point and a relative error of 2^-28 at most, mostly of random
// sign.  Sums are exact in any order: the result does not depend on how the row is split.
//
// One cluster per row, a CTA holds a run of 256-id tiles.  What a row's rules ask for decides its way:
//   k = 1 (or T = 0)      the largest logit's lowest id, found in the pass that finds the largest logit
//   k up to 1024          that pass keeps the largest of each of 4096 groups of ids; the k-th largest of those is
//                         no larger than the k-th logit, and few logits above it are not among the k.  These come
//                         together, in order of their ids, in the first CTA, which puts them into classes and finishes
//   a least share         is a least logit (a comparison); if few ids reach it they are finished in the same way
//   p alone               the weights of 2048 classes of (max - l) / T, the border class's ids as above; then the
//                         kept weight of every tile, and the one tile that holds the draw once more
//   other k, many equals  the same with counts (weights) of the key's leading bits, then of the border class's next
// Few rows are bound by the chain of passes and of the cluster's meetings, many by the weights (about 30
// instructions) and the classes' atomics.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_sample;
static std::atomic<bool> g_used_sample{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_sample() { return g_used_sample ? take_word(g_err_sample) : 0u; }

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 256;                   // ids a warp takes at once, eight a lane
constexpr int kMaxTiles = 512;               // of a CTA
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kScale = 42;                   // a weight of 1 is 2^42: 2^20 of them stay below 2^63
constexpr int kList = 2048;                  // ids that one CTA finishes
constexpr int kSmallK = 1024;
constexpr int kClasses = kThreads;           // of a list
constexpr int kMembers = 256;                // ids of a class that are compared one by one
constexpr int kStage = kList / kWarps;       // ids that a warp holds before it knows their places
constexpr int kGroups = 4096;                // groups whose largest logits bound the k-th: eight a thread at most

struct Find {           // where the order's prefix ends: in this class,
  u64 above;            // after so many ids (so much weight) of the classes above it,
  u64 in;               // with so much in it
  uint32_t bin;
};
struct Shared {
  union {
    struct {
      uint32_t cnt[kBins];                   // ids in a class, and
      union {
        u64 sum[kBins];                      // their weights, or
        uint32_t part[2][kBins];             // of their lower and upper halves
      };
    };
    u64 order[kList];                        // ids on their way to a list; a list's sort keys
    struct {
      u64 member[kMembers], member_weight[kMembers], before[kMembers];
    };
  };
  union {
    struct {
      uint32_t key[kList];                   // a list's keys and ids, in order of the ids
      int32_t id[kList];
    };
    uint32_t group[kGroups];                 // the largest key of each group of ids
  };
  u64 tile_mass[kMaxTiles];                  // kept weight of a tile (ties: how many)
  uint2 table[32];                           // 2^31 2^(j / 32), and the same in fp32
  u64 warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  // written by the cluster's CTAs, one entry each
  u64 part_mass[kMaxCluster];
  uint32_t part_count[kMaxCluster];
  float part_max[kMaxCluster];
  Find found;
  uint32_t members;
  uint32_t cutoff, border;
  float least;
  double least_off;      // T ln of the least share
  float near_off;        // the same in fp32 (that conversion by all threads took 2 us)
};

// order of values as order of unsigned integers; bf16 values use the upper half
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 counts as +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }
template <typename T>
__device__ __forceinline__ uint32_t key_of(float v) {
  return sizeof(T) == 2 ? ordered(v) >> 16 : ordered(v);
}
template <typename T>
__device__ __forceinline__ float value_of(uint32_t key) {
  return unordered(sizeof(T) == 2 ? key << 16 | ((key & 0x8000u) ? 0u : 0xffffu) : key);
}

struct Heat {
  float mx, ch, cl;      // the largest logit; log2(e) / T as two fp32 parts
};
// acc + 2^42 exp((v - mx) / T).  y = (v - mx) log2(e) / T comes as two parts, k / 32 nearest to it is taken out
// exactly, and 2^r - 1 of the rest (at most 1/64) multiplies a table's 2^(k mod 32 / 32): w with 31 bits behind the
// point.  What lies 2^-42 below the largest weighs nothing.
__device__ __forceinline__ uint32_t shift_right(uint32_t x, int n) {      // n from 0 on; 32 and more give 0
  uint32_t y;
  asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(n));
  return y;
}
// w = 2^(k mod 32 / 32) 2^r with 31 bits behind the point, and 0x4B400000 + k
template <typename T>
__device__ __forceinline__ uint32_t mantissa(float v, const Heat& h, const uint2* table, uint32_t& bits) {
  const float d = v == h.mx ? 0.f : v - h.mx;          // (two infinities have no difference)
  float lo;                                            // what the product loses, and the difference before it (of
  const float y = d * h.ch;                            // bf16 values: nothing that matters)
  if (sizeof(T) == 4) {
    const float b = d - v, e = (v - (d - b)) + (-h.mx - b);
    lo = fmaf(d, h.ch, -y) + fmaf(d, h.cl, e * h.ch);
  } else {
    lo = fmaf(d, h.cl, fmaf(d, h.ch, -y));
  }
  const float yc = fmaxf(y, -60.0f);                   // (2^-60 is none; a lo that is no number then does not matter)
  const float kf = fmaf(yc, 32.0f, 12582912.0f);
  bits = __float_as_uint(kf);
  const float r = fmaf(kf - 12582912.0f, -0.03125f, yc) + lo;
  // (ln 2)^n / n!
  const float E = r * fmaf(r, fmaf(r, fmaf(r, 9.6181291e-3f, 5.5504109e-2f), 2.4022651e-1f), 6.9314718e-1f);
  const uint2 t = table[bits & 31];
  return t.x + (uint32_t)__float2int_rn(__uint_as_float(t.y) * E);
}
// how far w is shifted up (down) to the scale of the sums
__device__ __forceinline__ int shift_of(uint32_t bits) { return ((int)(bits - 0x4B400000u) >> 5) + (kScale - 31); }
template <typename T>
__device__ __forceinline__ u64 add_weight(u64 acc, float v, const Heat& h, const uint2* table) {
  uint32_t bits;
  const uint32_t w = mantissa<T>(v, h, table, bits);
  const int up = shift_of(bits);
  return acc + (u64)shift_right(w, max(-up, 0)) * (u64)(1u << max(up, 0));
}
template <typename T>
__device__ __forceinline__ u64 weight(float v, const Heat& h, const uint2* table) {
  return add_weight<T>(0ull, v, h, table);
}
// The class of a logit by its k, larger for a larger one: 32 to an octave of weight.  In a class all w have one shift.
__device__ __forceinline__ uint32_t class_at(uint32_t bits) { return kBins - 1 + (bits - 0x4B400000u); }
__device__ __forceinline__ uint32_t class_of(float v, const Heat& h) {
  const float d = v == h.mx ? 0.f : v - h.mx;
  return class_at(__float_as_uint(fmaf(fmaxf(d * h.ch, -60.0f), 32.0f, 12582912.0f)));
}
// ln(exp((v - mx) / T) / total), total in units of 2^-42, rounded about once: q = (v - mx) / T and e ln 2 as two
// parts, ln m of total = m 2^e as logf's value and what exp of that is off by.  (In fp64 the one thread that does
// this took a microsecond.)
__device__ __forceinline__ float log_share(float v, const Heat& h, float T, u64 total, const uint2* table) {
  float d = 0.f, dl = 0.f;
  if (v != h.mx) {
    d = v - h.mx;
    const float b = d - v;
    dl = (v - (d - b)) + (-h.mx - b);
  }
  const float q = d / T, ql = (fmaf(-q, T, d) + dl) / T;
  const int z = __clzll((long long)total), e = 63 - z - kScale;
  const u64 m = total << z;                                            // m / 2^63 in [1, 2)
  const float mf = (float)(uint32_t)(m >> 40) * 1.1920929e-7f, y = logf(mf);
  // 2^x, x = -y log2(e), as above: w 2^(k >> 5)
  const float x = -y * 1.44269502f, xl = fmaf(-y, 1.44269502f, -x) - y * 1.92596303e-8f;
  const float kf = fmaf(x, 32.0f, 12582912.0f);
  const uint32_t bits = __float_as_uint(kf);
  const float r = fmaf(kf - 12582912.0f, -0.03125f, x) + xl;
  const float E = r * fmaf(r, fmaf(r, fmaf(r, 9.6181291e-3f, 5.5504109e-2f), 2.4022651e-1f), 6.9314718e-1f);
  const uint2 t = table[bits & 31];
  const uint32_t w = t.x + (uint32_t)__float2int_rn(__uint_as_float(t.y) * E);
  // m w 2^(k >> 5) is near 1 (2^62 as the upper half of the product counts, k >> 5 is 0 or -1): what it is off by
  const u64 one = __umul64hi(m, (u64)w << 32) >> -((int)(bits - 0x4B400000u) >> 5);
  const float off = (float)(int64_t)(one - (1ull << 62)) * 2.16840434e-19f;
  const float eh = (float)e * 0.693145752f, el = (float)e * 1.42860677e-6f;    // ln 2: 16 bits, and the rest
  // -(q + ql) + eh + el + y + off, all of one sign but the small ones
  const float s1 = eh - q, b1 = s1 - eh, e1 = (eh - (s1 - b1)) + (-q - b1);
  const float s2 = s1 + y, b2 = s2 - s1, e2 = (s1 - (s2 - b2)) + (y - b2);
  return -(s2 + (e1 + e2 + el - ql + off));
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <typename V>
__device__ __forceinline__ V* at_rank(V* p, int rank) {      // the same object in another CTA of the cluster
  u64 a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<u64>(p)), "r"(rank));
  return reinterpret_cast<V*>(a);
}

// x in [0, 1) as a fraction of 2^64 (exact from 2^-40 on)
__device__ __forceinline__ u64 fraction(float x) {
  const uint32_t b = __float_as_uint(x);
  const int e = (int)(b >> 23) - 86;                                    // x = m 2^(e - 64)
  const u64 m = b < 0x00800000u ? 0ull : (b & 0x7fffffu) | 0x800000u;
  return e >= 0 ? m << e : (e > -24 ? m >> -e : 0ull);
}
// log2(e) / T as two fp32 parts (fp64 would do, at a sixtieth of the rate: 4 us for a CTA's threads)
__device__ __forceinline__ void heat_parts(float T, Heat& h) {
  const float hi = 1.44269502f, lo = 1.92596303e-8f;                    // log2(e)
  h.ch = hi / T;
  h.cl = isinf(h.ch) ? 0.f : (fmaf(-h.ch, T, hi) + lo) / T;
}

// ceil(a share of `of`), at least 1; the share as a fraction of 2^64
__device__ __forceinline__ u64 share_of(u64 of, u64 share) {
  const u64 t = __umul64hi(of, share) + (of * share != 0);
  return t ? t : 1ull;
}

struct Rules {
  uint32_t k;            // 1..; 0xffffffff: all
  u64 p;                 // the share as a fraction of 2^64 (p_on)
  bool p_on;
  float least;           // the least logit kept
  u64 u;
  float heat;            // > 0
};

struct Args {
  int32_t* token;
  float* logprob;
  int32_t* kept;
  const float* u;
  cb_sample_rules r;
  int vocab, tpc;
  bool vec;
};

// One row's work as its cluster sees it.
template <typename T>
struct Row {
  static constexpr int kKey = sizeof(T) == 2 ? 16 : 32;
  const T* x;
  Shared* s;
  Heat heat;
  int vocab, tile0, tiles, nc, rank;
  bool vec;

  __device__ __forceinline__ void meet() const {             // everything written so far is seen by the whole cluster
    if (nc > 1)
      tc::cluster_sync();
    else
      __syncthreads();
  }
  __device__ __forceinline__ Shared* at(int q) const { return nc > 1 ? at_rank(s, q) : s; }
  // the lane's eight values of tile t of this CTA; past the end -inf
  __device__ __forceinline__ int load(int t, float* f) const {
    const int lane = threadIdx.x & 31, id = (tile0 + t) * kTile + lane * 8;
    if (vec && id + 8 <= vocab) {
      ld8(x + id, f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = id + i < vocab ? to_f(x[id + i]) : -INFINITY;
    }
    return id;
  }
  // fn(first id of the lane's eight, the eight, tile) for tiles t0, t0 + step, ... below t1, four loads in flight
  template <typename Fn>
  __device__ __forceinline__ void each(int t0, int t1, int step, Fn fn) const {
    constexpr int U = sizeof(T) == 2 ? 4 : 2, Q = sizeof(T) / 2;
    const int lane = threadIdx.x & 31;
    for (int t = t0; t < t1; t += U * step) {
      uint4 raw[U][Q];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tt = t + u * step, id = (tile0 + tt) * kTile + lane * 8;
        if (vec && tt < t1 && id + 8 <= vocab)
#pragma unroll
          for (int q = 0; q < Q; ++q) raw[u][q] = reinterpret_cast<const uint4*>(x + id)[q];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tt = t + u * step, id = (tile0 + tt) * kTile + lane * 8;
        if (tt >= t1) break;
        float f[8];
        if (vec && id + 8 <= vocab) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[u]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[i] = Q == 2 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = id + i < vocab ? to_f(x[id + i]) : -INFINITY;
        }
        fn(id, f, tt);
      }
    }
  }
  __device__ __forceinline__ u64 weigh(float v) const { return weight<T>(v, heat, s->table); }
  __device__ __forceinline__ u64 add(u64 acc, float v) const { return add_weight<T>(acc, v, heat, s->table); }

  // This CTA's exclusive sum over its threads, and the sum of all (every thread calls)
  __device__ __forceinline__ void scan(uint32_t& c, u64& m, uint32_t& ct, u64& mt) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ci = c;
    u64 mi = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, ci, o);
      const u64 d = __shfl_up_sync(0xffffffffu, mi, o);
      if (lane >= o) {
        ci += a;
        mi += d;
      }
    }
    __syncthreads();                         // (what was there is read)
    if (lane == 31) {
      s->warp_count[warp] = ci;
      s->warp_mass[warp] = mi;
    }
    __syncthreads();
    // (a lane for each warp's sums; of 64 bits 21 at a time, and no carry is lost)
    const uint32_t wc = lane < kWarps ? s->warp_count[lane] : 0u;
    const u64 wm = lane < kWarps ? s->warp_mass[lane] : 0ull;
    const bool before = lane < warp;
    ct = __reduce_add_sync(0xffffffffu, wc);
    ci += __reduce_add_sync(0xffffffffu, before ? wc : 0u);
    mt = 0;
#pragma unroll
    for (int i = 0; i < 63; i += 21) {
      const uint32_t part = (uint32_t)(wm >> i) & 0x1fffffu;
      mt += (u64)__reduce_add_sync(0xffffffffu, part) << i;
      mi += (u64)__reduce_add_sync(0xffffffffu, before ? part : 0u) << i;
    }
    c = ci - c;
    m = mi - m;
  }

  // The ids' classes cls(value, key), -1: none, and in them counts (KIND 0), sums of weights (1), or sums of weights
  // in the classes of class_of (2).  Then, in falling order of classes, the one in which the running count (weight)
  // reaches the target behind what lies `above` all of them; want(all of it) gives the target.
  //
  // 64-bit sums are slow atomics (37 cycles a warp); the weights of a class of KIND 2 have one shift and 32 bits, and
  // two 32-bit sums of their halves do for 2^16 ids a CTA.  Beyond, what these carry is counted.
  template <int KIND, typename Cls, typename Want>
  __device__ __forceinline__ Find find(u64 above, Cls cls, Want want) {
    const int tid = threadIdx.x, warp = tid >> 5;
    for (int i = tid; i < kBins; i += kThreads) {
      if (KIND != 1) s->cnt[i] = 0;
      if (KIND != 0) s->sum[i] = 0;
    }
    __syncthreads();
    each(warp, tiles, kWarps, [&](int, const float* f, int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!(f[i] > -INFINITY)) continue;
        const int b = cls(f[i], key_of<T>(f[i]));
        if (b < 0) continue;
        if (KIND == 0) atomicAdd(&s->cnt[b], 1u);
        if (KIND == 1) atomicAdd(&s->sum[b], weigh(f[i]));
        if (KIND == 2) {
          uint32_t bits;
          const uint32_t w = mantissa<T>(f[i], heat, s->table, bits);
          const uint32_t u = shift_right(w, max(-shift_of(bits), 0)), c = class_at(bits);
          if (tiles <= 65536 / kTile) {
            atomicAdd(&s->part[0][c], u & 0xffffu);
            atomicAdd(&s->part[1][c], u >> 16);
          } else {
            if (atomicAdd(&s->part[0][c], u & 0xffffu) > ~(u & 0xffffu)) atomicAdd(&s->cnt[c], 1u);
            if (atomicAdd(&s->part[1][c], u >> 16) > ~(u >> 16)) atomicAdd(&s->cnt[c], 0x10000u);
          }
        }
      }
    });
    meet();
    // this CTA's share of the classes, in falling order; a thread holds up to four neighbours
    constexpr int kOwn = kBins / kThreads;
    const int share = kBins / nc, per = share > kThreads ? share / kThreads : 1;
    u64 m[kOwn], ms = 0, mt;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      m[j] = 0;
      const int i = tid * per + j;
      if (j < per && i < share) {
        const int b = kBins - 1 - (rank * share + i);
        u64 c = 0;
        for (int q = 0; q < nc; ++q) {
          const Shared* o = at(q);
          if (KIND == 0) c += o->cnt[b];
          if (KIND == 1) m[j] += o->sum[b];
          if (KIND == 2) {
            const uint32_t carry = o->cnt[b];
            m[j] += ((u64)(carry >> 16) << 48) + ((u64)o->part[1][b] << 16) + ((u64)(carry & 0xffffu) << 32) + o->part[0][b];
          }
        }
        if (KIND == 0) m[j] = c;
        if (KIND == 2) m[j] <<= max(shift_of(0x4B400000u + (uint32_t)(b - (kBins - 1))), 0);
      }
      ms += m[j];
    }
    u64 mb = ms;
    uint32_t none = 0, nt;
    scan(none, mb, nt, mt);
    if (tid < nc) at(tid)->part_mass[rank] = mt;
    meet();
    // what lies above this thread's classes
    u64 all = 0;
    mb += above;
    for (int q = 0; q < nc; ++q) {
      all += s->part_mass[q];
      if (q < rank) mb += s->part_mass[q];
    }
    const u64 target = want(all);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      if (mb < target && target <= mb + m[j]) {
        const Find r{mb, m[j], (uint32_t)(kBins - 1 - (rank * share + tid * per + j))};
        for (int q = 0; q < nc; ++q) at(q)->found = r;
      }
      mb += m[j];
    }
    meet();
    return s->found;
  }

  // The ids with take(value) (false for -inf), in order, to the first CTA's list, if there are kList at most; how
  // many (the same in all CTAs), and the weight of all ids of the row where it is asked for.
  template <bool MASS, typename Take>
  __device__ __forceinline__ uint32_t gather(Take take, u64* weight_of_all) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tpw = (tiles + kWarps - 1) / kWarps, t0 = warp * tpw, t1 = min(tiles, t0 + tpw);
    u64* stage = s->order + warp * kStage;
    uint32_t found = 0;                      // of this warp
    u64 m = 0;
    // put(place among the warp's, key, id) for those taken
    auto walk = [&](auto put, bool mass) {
      found = 0;
      each(t0, t1, 1, [&](int id, const float* f, int) {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c += take(f[i]);
          if (MASS && mass && f[i] > -INFINITY) m = add(m, f[i]);
        }
        if (!__any_sync(0xffffffffu, c)) return;
        uint32_t incl = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += y;
        }
        uint32_t to = found + incl - c;
        if (c) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (take(f[i])) put(to++, key_of<T>(f[i]), id + i);
        }
        found += __shfl_sync(0xffffffffu, incl, 31);
      });
    };
    walk([&](uint32_t to, uint32_t key, int id) {
      if (to < kStage) stage[to] = (u64)key << 32 | (uint32_t)id;
    }, true);
    uint32_t before = lane ? 0 : found, ct;
    u64 mt;
    scan(before, m, ct, mt);
    if (tid < nc) {
      at(tid)->part_count[rank] = ct;
      if (MASS) at(tid)->part_mass[rank] = mt;
    }
    meet();
    uint32_t base = 0, total = 0;
    u64 all = 0;
    for (int q = 0; q < nc; ++q) {
      if (q < rank) base += s->part_count[q];
      total += s->part_count[q];
      if (MASS) all += s->part_mass[q];
    }
    if (MASS) *weight_of_all = all;
    if (total <= kList) {
      Shared* o = at(0);
      base += __shfl_sync(0xffffffffu, before, 0);
      auto put = [&](uint32_t to, uint32_t key, int id) {
        o->key[base + to] = key;
        o->id[base + to] = id;
      };
      if (found <= kStage) {
        for (uint32_t i = lane; i < found; i += 32) put(i, (uint32_t)(stage[i] >> 32), (int)(uint32_t)stage[i]);
      } else {
        walk(put, false);                    // more than there is room for: once more
      }
    }
    meet();
    return total;
  }

  // Sorts a list of n: order[r] is (all bits of the key inverted, place in the list), rising.  A warp owns 64
  // neighbours at a time, so that steps of up to 32 need no other warp.
  __device__ __forceinline__ void sort(int n) const {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int N = 64;
    while (N < n) N <<= 1;
    for (int i = tid; i < N; i += kThreads) s->order[i] = i < n ? (u64)~s->key[i] << 32 | (uint32_t)i : ~0ull;
    __syncthreads();
    auto step = [&](int i, int j, int size) {      // the pair (i, i + j)
      const u64 a = s->order[i], b = s->order[i + j];
      if ((a > b) == ((i & size) == 0)) {
        s->order[i] = b;
        s->order[i + j] = a;
      }
    };
    for (int size = 2; size <= N; size <<= 1) {
      int j = size >> 1;
      for (; j > 32; j >>= 1) {
        for (int q = tid; q < N / 2; q += kThreads) step((q & ~(j - 1)) * 2 + (q & (j - 1)), j, size);
        __syncthreads();
      }
      for (int w = warp * 64; w < N; w += kWarps * 64)
        for (int d = j; d > 0; d >>= 1) {
          step(w + (lane & ~(d - 1)) * 2 + (lane & (d - 1)), d, size);
          __syncwarp();
        }
      if (size >= 64) __syncthreads();
    }
    __syncthreads();
  }

  // Which of a list are among the first k of the order, and of those (p_on) come before a target of weight is reached,
  // with `above` before the list: `of`, or (above = 0) the share p of it, of the weight of the first k with of = 0.  The
  // id at which it is reached becomes border and cutoff; the others' ids get their top bit set.
  // Keys (bf16: there are few of them) or ranges of values are classes; only the ids of the class in which the order
  // ends are compared with one another, equals by counting.  With more than kMembers of them that are not equal the
  // list is sorted, which takes 12 us of a CTA for 2048 ids.
  // One CTA runs through this once a row, and instructions that it meets for the first time cost it more than what
  // they do: loops stay loops, and the first k and p go the same way (unrolled, k = 50 with p took 2 us more).
  __device__ __forceinline__ void select(int n, uint32_t k, bool p_on, u64 above, u64 of, u64 share) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (n + kThreads - 1) / kThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      lo = min(lo, s->key[i]);
      hi = max(hi, s->key[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    __syncthreads();                         // (what was there is read)
    if (lane == 0) {
      s->warp_count[warp] = lo;
      s->warp_mass[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, s->warp_count[lane % kWarps]);
    hi = __reduce_max_sync(0xffffffffu, (uint32_t)s->warp_mass[lane % kWarps]);
    const bool exact = hi - lo < kClasses;   // a class for every key
    const float vlo = value_of<T>(lo), scale = (float)(kClasses - 1) / (value_of<T>(hi) - vlo);
    auto class_in = [&](uint32_t key) -> int {           // (what is no number, with infinite ends, is class 0)
      return exact ? (int)(key - lo) : min(kClasses - 1, __float2int_rz((value_of<T>(key) - vlo) * scale));
    };
    bool few = true;
    uint32_t none = 0, no;
    u64 mt;
#pragma unroll 1
    for (int by = k < (uint32_t)n ? 0 : 1; by < (p_on ? 2 : 1); ++by) {      // by number, by weight
      auto amount = [&](uint32_t key) -> u64 { return by ? weigh(value_of<T>(key)) : 1ull; };
      s->sum[tid] = 0;
      if (tid == 0) s->members = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = i0; i < i1; ++i)
        if (s->id[i] >= 0) atomicAdd(&s->sum[class_in(s->key[i])], amount(s->key[i]));
      __syncthreads();
      const u64 m = s->sum[kClasses - 1 - tid], front = by ? above : 0ull;
      u64 mb = m;
      scan(none, mb, no, mt);
      none = 0;
      mb += front;
      const u64 limit = by ? (above ? of : share_of(of ? of : mt, share)) : (u64)k;
      if (limit > front + mt) break;         // all of them come before it
      if (mb < limit && limit <= mb + m) {
        s->found.bin = kClasses - 1 - tid;
        s->found.above = mb;
      }
      __syncthreads();
      const int b = (int)s->found.bin;
      const u64 base = s->found.above;
      auto decide = [&](int i, u64 at, u64 w) {          // `at` of the order lies before it
        if (at >= limit) {
          s->id[i] |= 0x80000000;
        } else if (by && limit <= at + w) {
          s->border = s->key[i];
          s->cutoff = s->id[i];
        }
      };
      uint32_t x = 0;
      if (exact) {
#pragma unroll 1
        for (int i = i0; i < i1; ++i) x += s->id[i] >= 0 && class_in(s->key[i]) == b;
        u64 zero = 0, z;
        scan(x, zero, no, z);
      }
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        if (s->id[i] < 0) continue;
        const uint32_t key = s->key[i];
        const int c = class_in(key);
        if (c < b) s->id[i] |= 0x80000000;
        if (c != b) continue;
        const u64 w = amount(key);
        if (exact) {
          decide(i, base + w * x++, w);
        } else {
          const uint32_t to = atomicAdd(&s->members, 1u);
          if (to < kMembers) {               // its place in the order: all bits of the key inverted, place in the list
            s->member[to] = (u64)~key << 32 | (uint32_t)i;
            s->member_weight[to] = w;
            s->before[to] = base;
          }
        }
      }
      __syncthreads();
      if (!exact) {
        const int many = (int)s->members, i = tid % kMembers;
        if (many > kMembers) {
          few = false;
          break;
        }
        if (i < many) {
          const u64 mine = s->member[i];
          u64 sum = 0;
          for (int y = tid / kMembers; y < many; y += kThreads / kMembers) sum += s->member[y] < mine ? s->member_weight[y] : 0ull;
          if (sum) atomicAdd(&s->before[i], sum);
        }
        __syncthreads();
        if (tid < many) decide((int)(uint32_t)s->member[tid], s->before[tid], s->member_weight[tid]);
        __syncthreads();
      }
    }
    if (few) return;
    __syncthreads();
    sort(n);
    u64 run = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      s->id[i] &= 0x7fffffff;
      if (i < k) run += weigh(value_of<T>(~(uint32_t)(s->order[i] >> 32)));
    }
    scan(none, run, no, mt);
    const u64 limit = p_on ? (above ? of : share_of(of ? of : mt, share)) : ~0ull;
    run += above;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int at = (int)(uint32_t)s->order[i];
      if (i >= k || run >= limit) {
        s->id[at] |= 0x80000000;
        continue;
      }
      const u64 w = weigh(value_of<T>(~(uint32_t)(s->order[i] >> 32)));
      if (limit <= run + w) {
        s->border = s->key[at];
        s->cutoff = s->id[at];
      }
      run += w;
    }
    __syncthreads();
  }

  // The first CTA's list of n to the row's token.  all: the weight that p is a share of; 0: of the k kept.
  __device__ __forceinline__ void finish(int n, const Rules& r, u64 all, const Args& a, int row) {
    const int tid = threadIdx.x, per = (n + kThreads - 1) / kThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    const uint32_t k = min(r.k, (uint32_t)n);
    if (r.p_on || k < (uint32_t)n) select(n, k, r.p_on, 0ull, all, r.p);
    uint32_t kept = 0, ct;
    u64 m = 0, mt;
    auto weight_at = [&](int i) -> u64 { return s->id[i] >= 0 && value_of<T>(s->key[i]) >= r.least ? weigh(value_of<T>(s->key[i])) : 0ull; };
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      kept += s->id[i] >= 0 && value_of<T>(s->key[i]) >= r.least;
      m += weight_at(i);
    }
    scan(kept, m, ct, mt);
    const u64 target = __umul64hi(mt, r.u);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const u64 w = weight_at(i);
      if (m <= target && target < m + w) emit(s->id[i], value_of<T>(s->key[i]), mt, r, a, row);
      m += w;
    }
    if (tid == 0 && a.kept) a.kept[row] = (int32_t)ct;
  }

  __device__ __forceinline__ void emit(int id, float v, u64 total, const Rules& r, const Args& a, int row) const {
    a.token[row] = id;
    if (a.logprob) a.logprob[row] = log_share(v, heat, r.heat, total, s->table);
  }

  // A key that is no larger than the k-th largest of the row's, from the largest of its groups (first CTA).
  __device__ __forceinline__ uint32_t bound(uint32_t k) {
    const int tid = threadIdx.x;
    uint32_t prefix = 0, above = 0;
    int upto = kKey, shift = kKey - kBits;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
      for (int i = tid; i < kBins; i += kThreads) s->cnt[i] = 0;
      __syncthreads();
      for (int i = tid; i < kGroups; i += kThreads) {
        const uint32_t g = s->group[i];
        if (g && (level == 0 || g >> upto == prefix)) atomicAdd(&s->cnt[g >> shift & (kBins - 1)], 1u);
      }
      __syncthreads();
      constexpr int kOwn = kBins / kThreads;
      uint32_t c[kOwn], cs = 0, ct;
      u64 m = 0, mt;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) cs += c[j] = s->cnt[kBins - 1 - (tid * kOwn + j)];
      uint32_t cb = cs;
      scan(cb, m, ct, mt);
      if (above + ct < k) return 0;          // fewer groups than k hold an id (uniform)
      cb += above;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        if (cb < k && k <= cb + c[j]) {
          s->found.bin = kBins - 1 - (tid * kOwn + j);
          s->found.above = cb;
          s->found.in = c[j];
        }
        cb += c[j];
      }
      __syncthreads();
      const int bits = upto - shift;
      prefix = prefix << bits | (s->found.bin & ((1u << bits) - 1));
      above = (uint32_t)s->found.above;
      // (a class's lower end will do if not many more than k groups reach it)
      if (shift == 0 || above + (uint32_t)s->found.in <= max(256u, k + k / 4)) return prefix << shift;
      upto = shift;
      shift = max(0, shift - kBits);
      __syncthreads();
    }
    return prefix << (kKey == 32 ? 10 : 0);      // after two levels
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const T* __restrict__ logits, const Args a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y;
  constexpr int kKey = Row<T>::kKey;
  if (tid < 32) {
    const double t = exp2(tid / 32.0);
    const uint32_t w = (uint32_t)(t * 2147483648.0 + 0.5);
    sh.table[tid] = make_uint2(w, __float_as_uint((float)(t * 2147483648.0)));
  }
  Row<T> R;
  R.x = logits + (int64_t)row * a.vocab;
  R.s = &sh;
  R.vocab = a.vocab;
  R.nc = gridDim.x;
  R.rank = blockIdx.x;
  R.vec = a.vec;
  const int all_tiles = (a.vocab + kTile - 1) / kTile;
  R.tile0 = R.rank * a.tpc;
  R.tiles = max(0, min(a.tpc, all_tiles - R.tile0));
  if (tid == 0) sh.members = 0;
  R.meet();                                  // every CTA of the cluster runs before its memory is written
  pdl_wait();
  pdl_trigger();
  const bool report = R.rank == 0 && tid == 0;

  // ---- the row's settings
  float heat = a.r.temperature ? a.r.temperature[row] : 1.0f;
  const int ask = a.r.top_k ? a.r.top_k[row] : 0;
  float p = a.r.top_p ? a.r.top_p[row] : 1.0f, mp = a.r.min_p ? a.r.min_p[row] : 0.0f, u = a.u[row];
  bool bad = isnan(p) || isnan(mp) || !(u >= 0.0f && u < 1.0f);
  if (!(heat >= 0.0f) || isinf(heat)) {
    bad = true;
    heat = 1.0f;
  }
  if (heat < 1.17549435e-38f) heat = 0.0f;             // (1 / T would be infinite)
  if (bad && report) atomicOr(&g_err_sample, ERRBIT_NONFINITE);
  if (isnan(p)) p = 1.0f;
  if (isnan(mp)) mp = 0.0f;
  if (!(u >= 0.0f)) u = 0.0f;
  if (u >= 1.0f) u = 0.99999994f;
  Rules r;
  r.k = heat == 0.0f ? 1u : (ask <= 0 ? 0xffffffffu : (uint32_t)ask);
  r.p_on = p < 1.0f && r.k > 1;
  r.p = fraction(fminf(fmaxf(p, 0.0f), 0.99999994f));
  r.u = fraction(u);
  r.heat = heat > 0.0f ? heat : 1.0f;
  const bool grouped = r.k > 1 && r.k <= kSmallK;
  if (mp > 0.0f && tid == kThreads - 32) {
    sh.least_off = (double)r.heat * log(fmin((double)mp, 1.0));
    sh.near_off = (float)sh.least_off;
  }

  // ---- the largest logit, how many there are, and the largest of each group
  float top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = -INFINITY;
  uint32_t n = 0;
  int first = 0x7fffffff;                    // the lowest id of the largest one (k = 1)
  bool nan = false;
  if (r.k == 1) {
    R.each(warp, R.tiles, kWarps, [&](int id, const float* f, int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (f[i] > top[0]) {                 // (ids rise from tile to tile and within a lane)
          top[0] = f[i];
          first = id + i;
        }
        nan |= f[i] != f[i];
      }
    });
    n = top[0] > -INFINITY;                  // (only whether there is one)
  } else {
    R.each(warp, R.tiles, kWarps, [&](int, const float* f, int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        nan |= f[i] != f[i];
        n += f[i] > -INFINITY;
        top[i] = fmaxf(top[i], f[i]);
      }
    });
  }
  if (nan) atomicOr(&g_err_sample, ERRBIT_NONFINITE);
  if (grouped) {
    // eight groups a thread in a cluster of one, four in one of two, ...: kGroups in all
    const int per = 8 / R.nc;
    uint32_t* to = (R.nc > 1 ? at_rank(sh.group, 0) : sh.group) + (R.rank * kThreads + tid) * per;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= per) break;
      float v = top[i];
#pragma unroll
      for (int j = 1; j < 8; ++j)
        if (i + j * per < 8) v = fmaxf(v, top[i + j * per]);
      to[i] = v > -INFINITY ? key_of<T>(v) : 0u;
    }
  }
  float mx = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
  u64 best = r.k == 1 && mx > -INFINITY ? (u64)ordered(mx) << 32 | (uint32_t)~first : 0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 y = __shfl_xor_sync(0xffffffffu, best, o);
    best = y > best ? y : best;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  mx = warp_max(mx);
  if (lane == 0) {
    sh.warp_count[warp] = n;
    sh.warp_mass[warp] = r.k == 1 ? best : (u64)__float_as_uint(mx);
  }
  __syncthreads();
  if (tid < R.nc) {
    n = 0;
    best = 0;
    for (int w = 0; w < kWarps; ++w) {
      n += sh.warp_count[w];
      if (r.k == 1)
        best = sh.warp_mass[w] > best ? sh.warp_mass[w] : best;
      else
        mx = fmaxf(mx, __uint_as_float((uint32_t)sh.warp_mass[w]));
    }
    Shared* o = R.at(tid);
    o->part_count[R.rank] = n;
    o->part_max[R.rank] = mx;
    o->part_mass[R.rank] = best;
  }
  R.meet();
  n = 0;
  best = 0;
  mx = -INFINITY;
  for (int q = 0; q < R.nc; ++q) {
    n += sh.part_count[q];
    mx = fmaxf(mx, sh.part_max[q]);
    best = sh.part_mass[q] > best ? sh.part_mass[q] : best;
  }
  if (n == 0 || r.k == 1) {                  // (uniform over the cluster, whose memory no one reads any more)
    if (report) {
      a.token[row] = n ? (int32_t)~(uint32_t)best : -1;
      if (a.logprob) a.logprob[row] = n ? 0.0f : -INFINITY;
      if (a.kept) a.kept[row] = n ? 1 : 0;
    }
    return;
  }
  R.heat.mx = mx;
  heat_parts(r.heat, R.heat);
  if (tid == 0) sh.least = mp > 0.0f ? __double2float_ru((double)mx + sh.least_off) : -INFINITY;
  if (r.k >= n) r.k = 0xffffffffu;
  if (r.k > n && mp > 0.0f && r.p_on) {      // how many groups reach the least share, about
    const float near = mx + sh.near_off;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) c += top[i] >= near;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) atomicAdd(&sh.members, c);
  }
  R.meet();                                  // what the CTAs told one another has been read
  r.least = sh.least;

  // ---- few ids: one CTA finishes
  u64 whole = 0;                             // the weight of all ids, where it is known
  if (grouped && r.k < n) {
    if (R.rank == 0) {
      const uint32_t b = R.bound(r.k);
      if (tid < R.nc) R.at(tid)->border = b;
    }
    R.meet();
    const float b = fmaxf(value_of<T>(sh.border), -3.40282347e38f);      // (key 0: all)
    const uint32_t held = R.template gather<false>([&](float v) { return v >= b; }, nullptr);
    if (held <= kList) {
      if (R.rank == 0) R.finish(held, r, 0ull, a, row);
      return;
    }
  }
  // (more groups than 1500 would be more ids than a list takes, and the weights of all ids are not worth the attempt: 256
  // rows of 131072, some so, 159 us with it, 126 without)
  uint32_t reach = 0;
  if (r.k > n && mp > 0.0f && r.p_on)
    for (int q = 0; q < R.nc; ++q) reach += R.at(q)->members;
  if (r.k > n && mp > 0.0f && reach <= 1500) {
    u64 all = 0;
    auto take = [&](float v) { return v >= r.least && v > -INFINITY; };
    const uint32_t held = r.p_on ? R.template gather<true>(take, &all) : R.template gather<false>(take, nullptr);
    if (held <= kList) {
      if (R.rank == 0) R.finish(held, r, all, a, row);
      return;
    }
    whole = all;
  }

  // ---- where the order's kept prefix ends: at the key `border`, of whose equals those up to the id `cutoff`
  uint32_t border = 0, cutoff = 0xffffffffu, quota = 0xffffffffu, ties = 0;
  // by the key's bits, of the ids that pick takes, with `above` before them
  auto descend = [&](auto kind, u64 above, auto pick, auto want) {
    constexpr bool M = decltype(kind)::value;
    Find f{above, 0, 0};
    uint32_t prefix = 0;
    int upto = 32, shift = kKey - kBits;
    u64 target = 0;
    for (;;) {
      f = R.template find<M ? 1 : 0>(
          f.above,
          [&](float v, uint32_t key) -> int {
            return pick(v, key) && (upto == 32 || key >> upto == prefix) ? (int)(key >> shift & (kBins - 1)) : -1;
          },
          [&](u64 all) { return target ? target : target = want(all); });
      const int bits = (upto == 32 ? kKey : upto) - shift;
      prefix = upto == 32 ? f.bin : prefix << bits | (f.bin & ((1u << bits) - 1));
      if (shift == 0) break;
      upto = shift;
      shift = max(0, shift - kBits);
    }
    border = prefix;
    const u64 each = M ? R.weigh(value_of<T>(border)) : 1ull;            // all of the last class are equal
    ties = (uint32_t)(f.in / each);
    quota = (uint32_t)((target - f.above + each - 1) / each);
  };
  if (r.k < n) descend(std::false_type{}, 0ull, [](float, uint32_t) { return true; }, [&](u64) { return (u64)r.k; });
  if (r.p_on) {
    const uint32_t floor = border;
    const u64 spare = quota < ties ? (u64)(ties - quota) * R.weigh(value_of<T>(border)) : 0ull;
    u64 target = 0;
    // (with the whole weight known the ids below the least share can be left out: a border among them is no border)
    const float from = fmaxf(floor ? value_of<T>(floor) : -3.40282347e38f, whole ? r.least : -3.40282347e38f);
    const Find f = R.template find<2>(
        0ull, [&](float v, uint32_t) -> int { return v >= from ? 0 : -1; },
        [&](u64 all) { return target = min(share_of(whole ? whole : all - spare, r.p), all); });
    auto in_class = [&](float v) { return v >= from && class_of(v, R.heat) == f.bin; };
    const uint32_t held = R.template gather<false>(in_class, nullptr);
    if (held <= kList) {
      if (R.rank == 0) {
        // (with nothing above the class the target is a share of 1 of it)
        R.select(held, held, true, f.above, target, ~0ull);
        __syncthreads();
        if (tid > 0 && tid < R.nc) {
          R.at(tid)->border = sh.border;
          R.at(tid)->cutoff = sh.cutoff;
        }
      }
      R.meet();
      border = sh.border;
      cutoff = sh.cutoff;
      quota = ties = 0;
    } else {
      descend(std::true_type{}, f.above, [&](float v, uint32_t) { return in_class(v); }, [&](u64) { return target; });
    }
  }

  // ---- equals at the border: the id up to which they are kept
  if (quota < ties) {
    for (int t = warp; t < R.tiles; t += kWarps) {
      float f[8];
      R.load(t, f);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m += f[i] > -INFINITY && key_of<T>(f[i]) == border;
      m = __reduce_add_sync(0xffffffffu, m);
      if (lane == 0) sh.tile_mass[t] = m;
    }
    __syncthreads();
    uint32_t mine = 0;
    for (int t = lane; t < R.tiles; t += 32) mine += (uint32_t)sh.tile_mass[t];
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (tid < R.nc) R.at(tid)->part_count[R.rank] = mine;
    R.meet();
    uint32_t before = 0;
    for (int q = 0; q < R.rank; ++q) before += sh.part_count[q];
    if (warp == 0 && before < quota && quota <= before + mine) {
      int t = 0;
      uint32_t run = before;
      for (; run + (uint32_t)sh.tile_mass[t] < quota; ++t) run += (uint32_t)sh.tile_mass[t];
      float f[8];
      const int id = R.load(t, f);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m += f[i] > -INFINITY && key_of<T>(f[i]) == border;
      uint32_t incl = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      uint32_t at = run + incl - m;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (f[i] > -INFINITY && key_of<T>(f[i]) == border && ++at == quota)
          for (int q = 0; q < R.nc; ++q) R.at(q)->cutoff = id + i;
    }
    R.meet();
    cutoff = sh.cutoff;
  }

  // ---- the kept weight of every tile: of the logits above `low`, and of those equal to it up to the id `upto`
  float low = border ? value_of<T>(border) : -INFINITY;
  int upto = border ? (int)min(cutoff, 0x7fffffffu) : -1;
  if (r.least > low) {
    low = r.least;
    upto = 0x7fffffff;
  }
  uint32_t kept = 0;
  R.each(warp, R.tiles, kWarps, [&](int id, const float* f, int t) {
    u64 m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (f[i] > low || (f[i] == low && id + i <= upto)) {
        m = R.add(m, f[i]);
        ++kept;
      }
    }
    m = warp_sum64(m);
    if (lane == 0) sh.tile_mass[t] = m;
  });
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (lane == 0) sh.warp_count[warp] = kept;
  __syncthreads();
  u64 mine = 0;
  for (int t = lane; t < R.tiles; t += 32) mine += sh.tile_mass[t];
  mine = warp_sum64(mine);
  if (tid < R.nc) {
    kept = 0;
    for (int w = 0; w < kWarps; ++w) kept += sh.warp_count[w];
    Shared* o = R.at(tid);
    o->part_mass[R.rank] = mine;
    o->part_count[R.rank] = kept;
  }
  R.meet();
  u64 before = 0, total = 0;
  kept = 0;
  for (int q = 0; q < R.nc; ++q) {
    if (q < R.rank) before += sh.part_mass[q];
    total += sh.part_mass[q];
    kept += sh.part_count[q];
  }
  if (report && a.kept) a.kept[row] = (int32_t)kept;
  const u64 target = __umul64hi(total, r.u);
  if (warp == 0 && before <= target && target < before + mine) {
    // the first tile whose end lies beyond the draw, 32 at a time
    int t = 0;
    u64 run = before;
    for (int t0 = 0;; t0 += 32) {
      const u64 w = t0 + lane < R.tiles ? sh.tile_mass[t0 + lane] : 0ull;
      u64 incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, target < run + incl);
      if (hit || t0 + 32 >= R.tiles) {
        const int who = hit ? __ffs(hit) - 1 : 0;
        t = t0 + who;
        run += __shfl_sync(0xffffffffu, incl - w, who);
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    float f[8];
    const int id = R.load(t, f);
    u64 w[8], m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m += w[i] = f[i] > low || (f[i] == low && id + i <= upto) ? R.weigh(f[i]) : 0ull;
    u64 incl = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    run += incl - m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (run <= target && target < run + w[j]) R.emit(id + j, f[j], total, r, a, row);
      run += w[j];
    }
  }
}

}  // namespace

template <typename T>
static cudaError_t launch_t(const void* logits, int n_rows, const Args& a, int nc, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, n_rows);
  cfg.blockDim = dim3(kThreads);
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
  return cudaLaunchKernelEx(&cfg, k_sample<T>, static_cast<const T*>(logits), a);
}

cudaError_t launch_sample(int dt, const void* logits, int n_rows, int vocab, const float* u, const cb_sample_rules& r,
                          int32_t* token, float* logprob, int32_t* kept, cudaStream_t s) {
  g_used_sample = true;
  Args a{token, logprob, kept, u, r, vocab, 0, vocab % 8 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0};
  const int tiles = (vocab + kTile - 1) / kTile;
  // As many CTAs as run at once (two an SM) with a tile for every warp, but two a row up to 304 rows: rows differ in
  // what they ask for, and the slowest counts.  8, 4, 2, 1 a row: one row of 32000 ids 12.0, 12.6, 14.8, 15.3 us; 64 of
  // 64000, some with a share alone, 42.9, 37.3, 48, 68; 256 of 131072 by different rules 173, 131, 126, 181, all by k = 50
  // and a share -, 68, 51, 36; 400 of 64000 by these -, 85, 61, 40.
  int nc = kMaxCluster;
  while (nc > 1 && tiles <= nc / 2 * kMaxTiles &&
         ((int64_t)(nc > 2 ? nc : 1) * n_rows > 304 || tiles < nc / 2 * kWarps))
    nc /= 2;
  a.tpc = (tiles + nc - 1) / nc;
  return dt == DT_BF16 ? launch_t<bf16>(logits, n_rows, a, nc, s) : launch_t<float>(logits, n_rows, a, nc, s);
}

}  // namespace cb
