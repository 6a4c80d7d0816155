// The next token of each row from given random numbers: temperature, the k largest, the fewest that hold
// a share p, a least share of the largest, then the draw, in one launch and without a sort.
//
//   w_i = exp((l_i - max) / T);  order: falling logit, then rising id
//   kept = the first k of the order; of them the fewest whose weight reaches p of theirs; of them w_i >= min_p
//   token = the first kept id (ascending) whose running weight exceeds u times the kept weight
//
// Every decision compares sums of weights, and it should be the one that 64-bit arithmetic takes: with
// fp32 weights a draw over 64000 near-equal ids would fall on another id in one row of fifty.  So a weight
// is an integer, 2^42 w: 2^x by a table of 32 steps and a polynomial of degree 4 on a remainder that holds
// 31 bits behind the point (relative error 2^-29 at most, mostly of random sign), and sums are exact in any
// order: the result does not depend on how the row is split.
//
// One cluster per row, a CTA holds a run of 256-id tiles.  Passes over the row (from L2 after the first):
// the largest logit; for k, counts of 2048 classes of the key's leading bits, then of the border class's next
// bits; for p the same with weights; where equal logits straddle the border, the id up to which they are kept;
// the kept weight of every tile; and the one tile that holds the draw once more.
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
constexpr int kPiece = 14;                   // bits of a weight's pieces in a class's sums: 2^17 of them fit 32 bits

struct Find {           // where the order's prefix ends: in this class, after so much of the classes above it
  u64 mass;             // weight above it
  uint32_t count;       // ids above it
  uint32_t in;          // ids in it
  u64 in_mass;          // their weight
  uint32_t bin;
};
struct Shared {
  uint32_t cnt[kBins];                       // of this CTA's ids in a class, and the pieces of their weights' sum
  uint32_t piece[3][kBins];
  u64 tile_mass[kMaxTiles];                  // kept weight of a tile (ties: how many)
  uint2 table[32];                           // 2^31 2^(j / 32), and the same in fp32
  u64 warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  // written by the cluster's CTAs, one entry each
  u64 part_mass[kMaxCluster];
  uint32_t part_count[kMaxCluster];
  float part_max[kMaxCluster];
  Find found;
  uint32_t cutoff;
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
// 2^42 exp((v - mx) / T).  y = (v - mx) log2(e) / T comes as two parts, k / 32 nearest to it is taken out
// exactly, and 2^r - 1 of the rest (at most 1/64) multiplies a table's 2^(k mod 32 / 32).
template <typename T>
__device__ __forceinline__ u64 weight(float v, const Heat& h, const uint2* table) {
  const float d = v - h.mx;
  float e = 0.f;                             // what the difference lost (of bf16 values: nothing that matters)
  if (sizeof(T) == 4) {
    const float b = d - v;
    e = (v - (d - b)) + (-h.mx - b);
  }
  const float y = d * h.ch;
  const float lo = fmaf(d, h.ch, -y) + fmaf(d, h.cl, e * h.ch);
  const float kf = fmaf(y, 32.0f, 12582912.0f);
  const int k = __float_as_int(kf) - 0x4B400000;
  const float r = fmaf(kf - 12582912.0f, -0.03125f, y) + lo;
  // (ln 2)^n / n!
  const float E = r * fmaf(r, fmaf(r, fmaf(r, 9.6181291e-3f, 5.5504109e-2f), 2.4022651e-1f), 6.9314718e-1f);
  const uint2 t = table[k & 31];
  const uint32_t w = t.x + (uint32_t)__float2int_rn(__uint_as_float(t.y) * E);
  const u64 full = ((u64)w << (kScale - 31)) >> (-(k >> 5) & 63);
  return v == h.mx ? 1ull << kScale : (y > -(kScale + 2.0f) ? full : 0ull);
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

// One row's work as its cluster sees it.
template <typename T>
struct Row {
  const T* x;
  Shared* s;
  Heat heat;
  int vocab, tile0, tiles, nc, rank;
  bool vec;

  __device__ void meet() const {             // everything written so far is seen by the whole cluster
    if (nc > 1)
      tc::cluster_sync();
    else
      __syncthreads();
  }
  // the lane's eight values of tile t of this CTA; past the end -inf
  __device__ int load(int t, float* f) const {
    const int lane = threadIdx.x & 31, id = (tile0 + t) * kTile + lane * 8;
    if (vec && id + 8 <= vocab) {
      ld8(x + id, f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = id + i < vocab ? to_f(x[id + i]) : -INFINITY;
    }
    return id;
  }

  // Counts (and weights) of the classes (key >> shift) & (kBins - 1) of the ids with key >> upto == prefix, and
  // key >= floor; upto 32: of all.  Then, in falling order of classes, the one in which the running count
  // (weight) reaches `target` behind what lies above the prefix.  want(total weight of the classes) gives the
  // target where it is not known before.
  template <bool MASS, typename Want>
  __device__ Find find(int shift, int upto, uint32_t prefix, uint32_t floor, Find above, Want want) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kBins; i += kThreads) {
      s->cnt[i] = 0;
      if (MASS) s->piece[0][i] = s->piece[1][i] = s->piece[2][i] = 0;
    }
    __syncthreads();
    for (int t = warp; t < tiles; t += kWarps) {
      float f[8];
      load(t, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t key = key_of<T>(f[i]);
        if (!(f[i] > -INFINITY) || key < floor || (upto < 32 && key >> upto != prefix)) continue;
        const uint32_t b = key >> shift & (kBins - 1);
        atomicAdd(&s->cnt[b], 1u);
        if (MASS) {
          const u64 w = weight<T>(f[i], heat, s->table);
          const uint32_t p0 = (uint32_t)w & ((1u << kPiece) - 1), p1 = (uint32_t)(w >> kPiece) & ((1u << kPiece) - 1),
                         p2 = (uint32_t)(w >> 2 * kPiece);
          if (p0) atomicAdd(&s->piece[0][b], p0);
          if (p1) atomicAdd(&s->piece[1][b], p1);
          if (p2) atomicAdd(&s->piece[2][b], p2);
        }
      }
    }
    meet();
    // this CTA's share of the classes, in falling order; a thread holds up to four neighbours
    constexpr int kPer = kBins / kThreads;
    const int share = kBins / nc, per = share > kThreads ? share / kThreads : 1;
    uint32_t c[kPer];
    u64 m[kPer];
    uint32_t cs = 0;
    u64 ms = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = 0;
      m[j] = 0;
      const int i = tid * per + j;
      if (j < per && i < share) {
        const int b = kBins - 1 - (rank * share + i);
        for (int q = 0; q < nc; ++q) {
          const Shared* o = nc > 1 ? at_rank(s, q) : s;
          c[j] += o->cnt[b];
          if (MASS)
            m[j] += (u64)o->piece[0][b] + ((u64)o->piece[1][b] << kPiece) + ((u64)o->piece[2][b] << 2 * kPiece);
        }
      }
      cs += c[j];
      ms += m[j];
    }
    uint32_t ci = cs;
    u64 mi = ms;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, ci, o);
      const u64 d = __shfl_up_sync(0xffffffffu, mi, o);
      if (lane >= o) {
        ci += a;
        mi += d;
      }
    }
    if (lane == 31) {
      s->warp_count[warp] = ci;
      s->warp_mass[warp] = mi;
    }
    __syncthreads();
    uint32_t ct = 0;
    u64 mt = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        ci += s->warp_count[w];
        mi += s->warp_mass[w];
      }
      ct += s->warp_count[w];
      mt += s->warp_mass[w];
    }
    if (tid < nc) {
      Shared* o = nc > 1 ? at_rank(s, tid) : s;
      o->part_count[rank] = ct;
      o->part_mass[rank] = mt;
    }
    meet();
    // what lies above this thread's classes
    u64 all = 0;
    uint32_t cb = above.count + ci - cs;
    u64 mb = above.mass + mi - ms;
    for (int q = 0; q < nc; ++q) {
      all += s->part_mass[q];
      if (q < rank) {
        cb += s->part_count[q];
        mb += s->part_mass[q];
      }
    }
    const u64 target = want(all);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const u64 before = MASS ? mb : cb, behind = MASS ? mb + m[j] : cb + c[j];
      if (before < target && target <= behind) {
        const Find r{mb, cb, c[j], m[j], (uint32_t)(kBins - 1 - (rank * share + tid * per + j))};
        for (int q = 0; q < nc; ++q) (nc > 1 ? at_rank(s, q) : s)->found = r;
      }
      cb += c[j];
      mb += m[j];
    }
    meet();
    return s->found;
  }
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

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(const T* __restrict__ logits, const Args a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y;
  constexpr int kKey = sizeof(T) == 2 ? 16 : 32;
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
  R.meet();                                  // every CTA of the cluster runs before its memory is written
  pdl_wait();
  pdl_trigger();
  const bool report = R.rank == 0 && tid == 0;

  // ---- the row's settings
  float heat = a.r.temperature ? a.r.temperature[row] : 1.0f;
  if (!(heat >= 0.0f) || isinf(heat)) {
    if (report) atomicOr(&g_err_sample, ERRBIT_NONFINITE);
    heat = 1.0f;
  }
  const int ask = a.r.top_k ? a.r.top_k[row] : 0;
  uint32_t k = heat == 0.0f ? 1u : (ask <= 0 ? 0xffffffffu : (uint32_t)ask);
  float p = a.r.top_p ? a.r.top_p[row] : 1.0f, mp = a.r.min_p ? a.r.min_p[row] : 0.0f, u = a.u[row];
  if (isnan(p) || isnan(mp) || !(u >= 0.0f && u < 1.0f)) {
    if (report) atomicOr(&g_err_sample, ERRBIT_NONFINITE);
    if (isnan(p)) p = 1.0f;
    if (isnan(mp)) mp = 0.0f;
    if (!(u >= 0.0f)) u = 0.0f;
    if (u >= 1.0f) u = 0.99999994f;
  }
  const u64 least = mp > 0.0f ? (u64)ceil(fmin((double)mp, 1.0) * (double)(1ull << kScale)) : 0ull;

  // ---- the largest logit, and how many there are
  float mx = -INFINITY;
  uint32_t n = 0;
  bool nan = false;
  for (int t = warp; t < R.tiles; t += kWarps) {
    float f[8];
    R.load(t, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      nan |= f[i] != f[i];
      n += f[i] > -INFINITY;
      mx = fmaxf(mx, f[i]);
    }
  }
  if (nan) atomicOr(&g_err_sample, ERRBIT_NONFINITE);
  n = __reduce_add_sync(0xffffffffu, n);
  mx = warp_max(mx);
  if (lane == 0) {
    sh.warp_count[warp] = n;
    sh.warp_mass[warp] = __float_as_uint(mx);
  }
  __syncthreads();
  if (tid < R.nc) {
    n = 0;
    for (int w = 0; w < kWarps; ++w) {
      n += sh.warp_count[w];
      mx = fmaxf(mx, __uint_as_float((uint32_t)sh.warp_mass[w]));
    }
    Shared* o = R.nc > 1 ? at_rank(&sh, tid) : &sh;
    o->part_count[R.rank] = n;
    o->part_max[R.rank] = mx;
  }
  R.meet();
  n = 0;
  mx = -INFINITY;
  for (int q = 0; q < R.nc; ++q) {
    n += sh.part_count[q];
    mx = fmaxf(mx, sh.part_max[q]);
  }
  if (n == 0) {                              // nothing above -inf (uniform over the cluster)
    if (report) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
      if (a.kept) a.kept[row] = 0;
    }
    R.meet();
    return;
  }
  const double c = 1.4426950408889634 / (double)(heat > 0.0f ? heat : 1.0f);
  R.heat = Heat{mx, (float)c, (float)(c - (double)(float)c)};
  R.meet();                                  // part_count and warp_count are used again

  // ---- where the order's kept prefix ends: at `border`, of whose equals the first `quota` by id count
  uint32_t border = 0, quota = 0xffffffffu, ties = 0;
  if (k == 1) {
    border = key_of<T>(mx);
    quota = 1;
    ties = 2;                                // (perhaps)
  } else {
    auto descend = [&](auto mass, uint32_t floor, auto want) {
      constexpr bool M = decltype(mass)::value;
      Find f{};
      uint32_t prefix = 0;
      int upto = 32, shift = kKey - kBits;
      u64 target = 0;
      for (;;) {
        f = R.template find<M>(shift, upto, prefix, floor, f, [&](u64 all) { return target ? target : target = want(all); });
        // (bits above the key's are 0; the class index keeps kBits bits, fewer where fewer are left)
        const int bits = (upto == 32 ? kKey : upto) - shift;
        prefix = upto == 32 ? f.bin : prefix << bits | (f.bin & ((1u << bits) - 1));
        if (shift == 0) break;
        upto = shift;
        shift = max(0, shift - kBits);
      }
      border = prefix;
      ties = f.in;
      // all of the last class are equal
      quota = M ? (uint32_t)((target - f.mass + f.in_mass / f.in - 1) / (f.in_mass / f.in)) : (uint32_t)(target - f.count);
    };
    if (k < n) descend(std::false_type{}, 0u, [&](u64) { return (u64)k; });
    if (p < 1.0f) {
      const u64 spare = quota < ties ? (u64)(ties - quota) * weight<T>(value_of<T>(border), R.heat, sh.table) : 0ull;
      const u64 share = p > 0.0f ? (u64)((double)p * 18446744073709551616.0) : 0ull;
      descend(std::true_type{}, border, [&](u64 all) -> u64 {
        const u64 of = all - spare, t = __umul64hi(of, share) + (of * share != 0);
        return t ? t : 1ull;
      });
    }
  }

  // ---- equals at the border: the id up to which they are kept
  uint32_t cutoff = 0xffffffffu;
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
    if (tid < R.nc) (R.nc > 1 ? at_rank(&sh, tid) : &sh)->part_count[R.rank] = mine;
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
          for (int q = 0; q < R.nc; ++q) (R.nc > 1 ? at_rank(&sh, q) : &sh)->cutoff = id + i;
    }
    R.meet();
    cutoff = sh.cutoff;
  }

  // ---- the kept weight of every tile
  auto kept_weight = [&](float v, int id) -> u64 {
    const uint32_t key = key_of<T>(v);
    if (!(v > -INFINITY) || key < border || (key == border && (uint32_t)id > cutoff)) return 0ull;
    return weight<T>(v, R.heat, sh.table);
  };
  uint32_t kept = 0;
  for (int t = warp; t < R.tiles; t += kWarps) {
    float f[8];
    const int id = R.load(t, f);
    u64 m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t key = key_of<T>(f[i]);
      if (!(f[i] > -INFINITY) || key < border || (key == border && (uint32_t)(id + i) > cutoff)) continue;
      const u64 w = weight<T>(f[i], R.heat, sh.table);
      if (w < least) continue;
      m += w;
      ++kept;
    }
    m = warp_sum64(m);
    if (lane == 0) sh.tile_mass[t] = m;
  }
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (lane == 0) sh.warp_count[warp] = kept;
  __syncthreads();
  u64 mine = 0;
  for (int t = lane; t < R.tiles; t += 32) mine += sh.tile_mass[t];
  mine = warp_sum64(mine);
  if (tid < R.nc) {
    kept = 0;
    for (int w = 0; w < kWarps; ++w) kept += sh.warp_count[w];
    Shared* o = R.nc > 1 ? at_rank(&sh, tid) : &sh;
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
  const u64 share = (u64)((double)u * 18446744073709551616.0), target = __umul64hi(total, share);
  if (warp == 0 && before <= target && target < before + mine) {
    int t = 0;
    u64 run = before;
    for (; run + sh.tile_mass[t] <= target; ++t) run += sh.tile_mass[t];
    float f[8];
    const int id = R.load(t, f);
    u64 w[8], m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = kept_weight(f[i], id + i);
      if (w[i] < least) w[i] = 0;
      m += w[i];
    }
    u64 incl = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    u64 at = run + incl - m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (at <= target && target < at + w[i]) {
        a.token[row] = id + i;
        if (a.logprob) {
          const double d = f[i] == mx ? 0.0 : (double)f[i] - (double)mx;
          a.logprob[row] = (float)(d / (double)(heat > 0.0f ? heat : 1.0f) - log((double)total / (double)(1ull << kScale)));
        }
      }
      at += w[i];
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
  int nc = kMaxCluster;
  while (nc > 1 && tiles <= nc / 2 * kMaxTiles && ((int64_t)nc * n_rows > 608 || tiles < nc * kWarps)) nc /= 2;
  a.tpc = (tiles + nc - 1) / nc;
  return dt == DT_BF16 ? launch_t<bf16>(logits, n_rows, a, nc, s) : launch_t<float>(logits, n_rows, a, nc, s);
}

}  // namespace cb
