// Attention over the 8-bit block-scaled KV cache (cb_kv8.cu), for a few query rows per KV head
// (single tokens) and, in tiles of 8 or 16 rows, for any number.
//
// With ks, vs the scales of key i's block and c_k, c_v its codes:
//   z_i = (q . c_k,i) * ks * log2(e) / sqrt(hd)                log2 of the unnormalised weight
//   out = sum_i 2^z_i vs c_v,i / sum_i 2^z_i
// The codes are small integers, exact in fp16, so they enter the matrix instructions as they
// are.  ks multiplies a score; vs is folded into the exponent: with t_i = z_i + log2 vs,
//   out = sum_i 2^(t_i - m) c_v,i / sum_i 2^(t_i - m) (1 / vs)
// for any reference m, kept near the largest t so far, which costs no extra multiplication
// and keeps the fp16 weights in range whatever the scales are.
//
// Rounding: q goes to fp16 after a division by a power of two per row (its 8 bf16 bits fit in
// fp16's 11; an element 2^14 below the row's largest loses bits that are 2^-25 of that
// largest), fp32 q as two such parts (22 bits).  2^(t - m) is rounded to fp16 (2^-11) beside
// the rounding of the bf16 output (2^-8), for fp32 output split in two parts.  Sums, maxima
// and accumulators are fp32.
#include <math.h>

#include <mutex>

#include "cb_kv8.cuh"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_kv8_attn;

uint32_t take_error_kv8_attn() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv8_attn, sizeof(v)) != cudaSuccess) return ERRBIT_INDEX;
  cudaMemcpyToSymbol(g_err_kv8_attn, &z, sizeof(z));
  return v;
}

namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr float kPBias = 8.0f;       // 2^(t - m) is held up to 2^8 ...
constexpr float kLazy = 6.0f;        // ... and up to 2^14 before m is raised: fp16 ends at 2^16
constexpr float kNone = -1e30f;      // m of a row that has seen no key
constexpr int MAX_SPLIT = 8;         // CTAs of a cluster

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t h2_sub1152(uint32_t x) {
  const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), k);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// codes 0,1 (lo) and 2,3 (hi) of a word as fp16 pairs: byte ^ 0x80 = c + 128, and 0x6400 | u
// is the fp16 number 1024 + u
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = h2_sub1152(__byte_perm(u, 0x64646464u, 0x4140));
  hi = h2_sub1152(__byte_perm(u, 0x64646464u, 0x4342));
}
// byte J of two words (two cache rows) as an fp16 pair
template <int J>
__device__ __forceinline__ uint32_t codes_pair(uint32_t a, uint32_t b) {
  const uint32_t x = __byte_perm(a, b, J | (J << 4) | ((4 + J) << 8) | ((4 + J) << 12));
  return h2_sub1152((x & 0x00ff00ffu) ^ 0x64806480u);
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

using tc::bulk_load;
using tc::ld_cluster;

// 8 x 8 transposition of fp16 pairs across the warp: thread (g, t) gives elements (g, 2t..2t+1)
// and gets (2t..2t+1, g)
__device__ __forceinline__ uint32_t transpose_h2(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

struct Kv8Attn {
  const void* q;
  const int32_t* last;      // [n_seq, n_q]
  void* out;
  float* z;                 // [n_seq * Hkv, n_q * G, capacity] scores z_i for the weights, or null
  float* lse;               // [n_seq, Hkv, n_q * G] log2 of a row's sum, or null
  float* weights;           // [n_seq, Hkv, capacity] (with z), or null
  cb_kv8_cache c;
  int n_q, H, Hkv, G, lg;
  float scale_log2;         // log2(e) / sqrt(hd)
};

// A stage holds KT keys, 16 KW per warp, so that its codes are 32 KB (64 KB at head_dim 256):
// three stages and two CTAs per SM (one at 256) keep about 190 KB of loads in flight per SM.
template <int HD>
struct Lay {
  static constexpr int KW = HD < 128 ? 128 / HD : 1;               // groups of 16 keys per warp and stage
  static constexpr int KT = 16 * WARPS * KW;
  static constexpr int HALF = KT * HD;                             // K (or V) codes of a stage
  static constexpr int NST = 3;
};
// shared memory of a CTA with row tiles of RT rows
template <int HD, int RT, bool QS, int NS>
struct Smem {
  using L = Lay<HD>;
  static constexpr int OFF_ML = L::NST * 2 * L::HALF;              // [2][WARPS][RT] row max and sum per warp
  static constexpr int OFF_CM = OFF_ML + 2 * WARPS * RT * 4;       // [RT] CTA max, [RT] CTA sum
  static constexpr int OFF_FM = OFF_CM + 2 * RT * 4;               // [RT] 1 / sum over the cluster, [RT] log2 of it
  static constexpr int OFF_LAST = OFF_FM + 2 * RT * 4;             // [RT]
  static constexpr int OFF_BAR = OFF_LAST + RT * 4;
  static constexpr int OFF_Q = (OFF_BAR + L::NST * 16 + 16 + 15) & ~15;   // fp16 q in fragment order (when not in registers)
  static constexpr int BYTES = OFF_Q + (QS ? NS * RT * HD * 2 : 0) + 128;
  static_assert(WARPS * RT * HD * 4 <= OFF_ML, "the merge buffer exceeds the stages");
  static_assert(MAX_SPLIT <= WARPS, "the factors of a cluster's CTAs reuse the warps' figures");
};
// fp16 parts of q and of the weights; whether q's fragments go to shared memory (two parts, or
// more than 32 registers)
template <typename T>
constexpr int parts() {
  return sizeof(T) == 4 ? 2 : 1;
}
template <int HD, int NT, typename T>
constexpr bool q_in_smem() {
  return parts<T>() == 2 || NT * (HD / 16) * 2 > 32;
}
template <int HD, int NT, typename T>
using SmemOf = Smem<HD, 8 * NT, q_in_smem<HD, NT, T>(), parts<T>()>;

template <typename T>
__device__ __forceinline__ void load4(const T* p, bool on, float* f) {
  if (on) {
    ld4(p, f);
  } else {
    f[0] = f[1] = f[2] = f[3] = 0.f;
  }
}

// One cluster of CTAs per (8 NT query rows, KV head, sequence); its CTAs take consecutive runs
// of the visible keys and are merged through distributed shared memory.  The products are
// taken transposed, S^T = C_K Q^T and O^T = C_V^T P^T, with the keys (then the channels) as
// the 16 rows of mma.m16n8k16 and the query rows as its 8 columns: the few rows of a single
// token fill the instruction (with rows as M, one token of grouped heads leaves more than half
// of the products, accumulators and conversions' consumers empty), and a thread's share of O
// is HD / 4 NT registers, which lets 16 warps live on an SM and hide each other's latencies.
// There is no producing warp: whichever warp is the last to finish a stage refills it.
// Measured before (rows as M, 10 warps per SM): 32 sequences of up to 16384 rows, 8 heads of
// 128, 205 us = 4.1 TB/s at an issue rate of 0.33 per scheduler.
template <int HD, int NT, typename T>
__global__ void __launch_bounds__(THREADS, HD == 256 ? 1 : 2) k_kv8_attn(const Kv8Attn p, int n_split) {
  pdl_wait();
  pdl_trigger();
  using L = Lay<HD>;
  using M = SmemOf<HD, NT, T>;
  constexpr int NS = parts<T>();
  constexpr bool QS = q_in_smem<HD, NT, T>();
  constexpr int KS = HD / 16;                    // k steps of a score; also channel tiles of O
  constexpr int RT = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((128 - (tc::smem_u32(smem_raw) & 127)) & 127);
  float* ml = reinterpret_cast<float*>(base + M::OFF_ML);
  float* cm = reinterpret_cast<float*>(base + M::OFF_CM);
  float* fm = reinterpret_cast<float*>(base + M::OFF_FM);
  int* slast = reinterpret_cast<int*>(base + M::OFF_LAST);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + M::OFF_BAR);
  uint32_t* spent = reinterpret_cast<uint32_t*>(full + L::NST);    // [NST] warps that have finished a stage, so far
  uint32_t* issued = spent + L::NST;                               // stages filled so far (valid once a wait has failed)
  uint32_t* failed = issued + 1;
  uint2* sq = reinterpret_cast<uint2*>(base + M::OFF_Q);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % n_split, rt = blockIdx.x / n_split, h = blockIdx.y, s = blockIdx.z;
  const int R = p.n_q * p.G, row0 = rt * RT, nrow = min(RT, R - row0);
  const int64_t cap = p.c.capacity, head = (int64_t)s * p.Hkv + h;

  if (tid < RT) {
    int l = -1;
    if (tid < nrow) {
      l = p.last[(int64_t)s * p.n_q + (row0 + tid) / p.G];
      if (l < -1 || l >= cap) {
        atomicOr(&g_err_kv8_attn, ERRBIT_INDEX);
        l = -1;
      }
    }
    slast[tid] = l;
  }
  if (tid == 0) {
    for (int i = 0; i < L::NST; ++i) {
      tc::mbar_init(&full[i], 1);
      spent[i] = 0;
    }
    *failed = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  int mx = -1, mn = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    mx = max(mx, slast[i]);
    if (i < nrow) mn = min(mn, slast[i]);
  }
  const int64_t nk = (int64_t)mx + 1;                        // keys some row sees
  const int tiles = (int)((nk + L::KT - 1) / L::KT);
  const int t0 = (int)((int64_t)tiles * rank / n_split), t1 = (int)((int64_t)tiles * (rank + 1) / n_split);

  float O[KS][NT][4];                            // channel tile, row tile: rows 2t, 2t + 1 of channels g, g + 8
  float m_used[NT][2], l_sum[NT][2];             // of rows 8 n + 2t, 2t + 1 (l: this thread's keys)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m_used[n][c] = kNone;
      l_sum[n][c] = 0.f;
    }
  bool ok = true;

  const int64_t nblk = cap >> p.lg;
  const float* ksc = p.c.k_scale + head * nblk;
  const float* vsc = p.c.v_scale + head * nblk;
  // fills stage u % NST with key tile t0 + u (one thread)
  auto fill = [&](int u) {
    const int st = u % L::NST;
    const int64_t k0 = (int64_t)(t0 + u) * L::KT, at = (head * cap + k0) * HD;
    const uint32_t bytes = (uint32_t)(cap - k0 < L::KT ? cap - k0 : L::KT) * HD;
    *issued = u + 1;
    tc::mbar_expect_tx(&full[st], 2 * bytes);
    bulk_load(base + st * 2 * L::HALF, p.c.k_codes + at, bytes, &full[st]);
    bulk_load(base + st * 2 * L::HALF + L::HALF, p.c.v_codes + at, bytes, &full[st]);
  };
  if (tid == 0)
    for (int u = 0; u < L::NST && u < t1 - t0; ++u) fill(u);

  {
    // Q^T as the column operand: thread (g, t) holds row 8 n + g, channels [t HD/4, (t + 1) HD/4),
    // 4 per k step (the order of the channels inside a sum is free; K is read with the same one)
    uint2 qb[QS ? 1 : NT][QS ? 1 : KS];
    float rf_g[NT];                                           // score factor of row 8 n + g
    {
      const T* q = static_cast<const T*>(p.q);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + g;
        const bool on = 8 * n + g < nrow;
        const int j = on ? r / p.G : 0;
        const T* qr = q + (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (on ? r - j * p.G : 0)) * HD + t * (HD / 4);
        float amax = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          float f[4];
          load4(qr + 4 * ks, on, f);
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e <= amax < 2^(e + 1); both powers stay normal
        int e = amax > 0.f ? ilogbf(amax) : 0;
        e = e < -120 ? -120 : (e > 120 ? 120 : e);
        const float down = ldexpf(1.0f, -e);
        rf_g[n] = ldexpf(p.scale_log2, e);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          float f[4];
          load4(qr + 4 * ks, on, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] *= down;
          const uint2 a = make_uint2(pack_h2(f[0], f[1]), pack_h2(f[2], f[3]));
          if constexpr (QS) {
            if (warp == 0) {
              sq[(n * KS + ks) * 32 + lane] = a;
              if constexpr (NS == 2)
                sq[((NT + n) * KS + ks) * 32 + lane] = make_uint2(rest_h2(f[0], f[1], a.x), rest_h2(f[2], f[3], a.y));
            }
          } else {
            qb[n][ks] = a;
          }
        }
      }
      if constexpr (QS) asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
    }
    float rf[NT][2];                                          // of rows 8 n + 2t, 2t + 1
    int lastr[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        rf[n][c] = __shfl_sync(0xffffffffu, rf_g[n], (2 * t + c) * 4);
        lastr[n][c] = slast[8 * n + 2 * t + c];
      }
    float* z = p.z ? p.z + (head * R + row0) * cap : nullptr;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) O[i][n][c] = 0.f;

    // scales of this warp's next 16 keys, loaded one step ahead (1 past the visible keys: their
    // block may never have been written)
    auto scales_of = [&](int64_t key) -> float2 {
      return key < nk ? make_float2(ksc[key >> p.lg], vsc[key >> p.lg]) : make_float2(1.0f, 1.0f);
    };
    float2 next = scales_of((int64_t)t0 * L::KT + warp * L::KW * 16);
    for (int j = t0; j < t1; ++j) {
      const int u = j - t0, st = u % L::NST;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[st], (u / L::NST) & 1));
      if (!ok) break;
      const uint8_t* sk = base + st * 2 * L::HALF;
#pragma unroll 1
      for (int w = 0; w < L::KW; ++w) {
        const int grp = warp * L::KW + w;
        const int64_t key0 = (int64_t)j * L::KT + grp * 16;
        const float2 cur = next;
        next = scales_of(w + 1 < L::KW ? key0 + 16 : key0 + L::KT - 16 * (L::KW - 1));
        if (key0 >= nk) continue;
        // ---- scores of 16 keys: thread (g, t) reads keys g and g + 8
        float S[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) S[n][c] = 0.f;
        const uint8_t* kr = sk + (grp * 16 + g) * HD + t * (HD / 4);
        constexpr int KC = HD >= 64 ? 16 : 8;                 // bytes per load
#pragma unroll
        for (int c0 = 0; c0 < HD / 4; c0 += KC) {
          uint32_t w0[KC / 4], w1[KC / 4];
          if constexpr (KC == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(kr + c0), y = *reinterpret_cast<const uint4*>(kr + 8 * HD + c0);
            w0[0] = x.x; w0[1] = x.y; w0[2] = x.z; w0[3] = x.w;
            w1[0] = y.x; w1[1] = y.y; w1[2] = y.z; w1[3] = y.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(kr + c0), y = *reinterpret_cast<const uint2*>(kr + 8 * HD + c0);
            w0[0] = x.x; w0[1] = x.y;
            w1[0] = y.x; w1[1] = y.y;
          }
#pragma unroll
          for (int i = 0; i < KC / 4; ++i) {
            const int ks = c0 / 4 + i;
            uint32_t a[4];                                    // rows g, g + 8 of channels 4 ks .. + 1, then + 2 .. + 3
            codes_to_h2(w0[i], a[0], a[2]);
            codes_to_h2(w1[i], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if constexpr (QS) {
#pragma unroll
                for (int part = 0; part < NS; ++part) {
                  const uint2 b = sq[((part * NT + n) * KS + ks) * 32 + lane];
                  mma_f16(S[n], a, b.x, b.y);
                }
              } else {
                mma_f16(S[n], a, qb[n][ks].x, qb[n][ks].y);
              }
            }
          }
        }
        // ---- weights: element c of S[n] is key g + 8 (c / 2), row 8 n + 2t + c % 2
        const float vs = fmaxf(cur.y, kKv8MinScale);
        const float3 sc = make_float3(fmaxf(cur.x, kKv8MinScale), NS == 2 ? log2f(vs) : __log2f(vs), __frcp_rn(vs));   // ks, log2 vs, 1 / vs
        const bool whole = key0 + 15 <= mn;                   // every row sees every key
        float f[NT][2], add[NT][2], e[NT][4];
        bool up = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            f[n][c] = rf[n][c] * sc.x;
            add[n][c] = sc.y - m_used[n][c] + kPBias;
          }
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if ((int)key0 + g + 8 * (c >> 1) > lastr[n][c & 1]) S[n][c] = -INFINITY;
          }
          if (z) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (8 * n + 2 * t + (c & 1) < nrow)
                z[(8 * n + 2 * t + (c & 1)) * cap + key0 + g + 8 * (c >> 1)] = S[n][c] * f[n][c & 1];
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            e[n][c] = fmaf(S[n][c], f[n][c & 1], add[n][c & 1]);
            up |= e[n][c] > kPBias + kLazy;
          }
        }
        // m is raised when a weight would leave fp16's range (and at a row's first key)
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float al[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float tt = fmaxf(S[n][c], S[n][c + 2]) * f[n][c];
              tt = fmaxf(tt, __shfl_xor_sync(0xffffffffu, tt, 4));
              tt = fmaxf(tt, __shfl_xor_sync(0xffffffffu, tt, 8));
              tt = fmaxf(tt, __shfl_xor_sync(0xffffffffu, tt, 16)) + sc.y;
              const bool raise = tt > m_used[n][c] + kLazy;
              al[c] = raise ? tc::ex2_approx(m_used[n][c] - tt) : 1.0f;
              if (raise) m_used[n][c] = tt;
              l_sum[n][c] *= al[c];
              add[n][c] = sc.y - m_used[n][c] + kPBias;
              e[n][c] = fmaf(S[n][c], f[n][c], add[n][c]);
              e[n][c + 2] = fmaf(S[n][c + 2], f[n][c], add[n][c]);
            }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
              for (int c = 0; c < 4; ++c) O[i][n][c] *= al[c & 1];
          }
        }
        uint32_t pb[NT][NS][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c = 0; c < 4; ++c) e[n][c] = tc::ex2_approx(e[n][c]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a = pack_h2(e[n][2 * k], e[n][2 * k + 1]);
            pb[n][0][k] = transpose_h2(a);
            if constexpr (NS == 2) pb[n][1][k] = transpose_h2(rest_h2(e[n][2 * k], e[n][2 * k + 1], a));
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) l_sum[n][c] = fmaf(e[n][c] + e[n][c + 2], sc.z, l_sum[n][c]);
        }
        // ---- O^T += C_V^T P^T: this thread's V rows are keys 2t, 2t+1, 2t+8, 2t+9; rows g, g + 8
        // of channel tile i stand for channels (HD/8) g + 2 i, + 1
        const uint8_t* vr = sk + L::HALF + (grp * 16 + 2 * t) * HD + g * (HD / 8);
        constexpr int VC = HD >= 128 ? 16 : HD / 8;           // bytes per load
#pragma unroll
        for (int c0 = 0; c0 < HD / 8; c0 += VC) {
          uint32_t v[4][VC / 4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint8_t* a = vr + ((r & 1) + 8 * (r >> 1)) * HD + c0;
            if constexpr (VC == 16) {
              const uint4 x = *reinterpret_cast<const uint4*>(a);
              v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
            } else if constexpr (VC == 8) {
              const uint2 x = *reinterpret_cast<const uint2*>(a);
              v[r][0] = x.x; v[r][1] = x.y;
            } else {
              v[r][0] = *reinterpret_cast<const uint32_t*>(a);
            }
          }
#pragma unroll
          for (int c = 0; c < VC / 4; ++c) {
            const uint32_t a0[4] = {codes_pair<0>(v[0][c], v[1][c]), codes_pair<1>(v[0][c], v[1][c]),
                                    codes_pair<0>(v[2][c], v[3][c]), codes_pair<1>(v[2][c], v[3][c])};
            const uint32_t a1[4] = {codes_pair<2>(v[0][c], v[1][c]), codes_pair<3>(v[0][c], v[1][c]),
                                    codes_pair<2>(v[2][c], v[3][c]), codes_pair<3>(v[2][c], v[3][c])};
            const int i = c0 / 2 + 2 * c;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int part = 0; part < NS; ++part) {
                mma_f16(O[i][n], a0, pb[n][part][0], pb[n][part][1]);
                mma_f16(O[i + 1][n], a1, pb[n][part][0], pb[n][part][1]);
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        // every warp's reads of the stage come before its count, the refill after the last one
        uint32_t before;
        asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(before) : "r"(tc::smem_u32(&spent[st])) : "memory");
        if (before == (uint32_t)(u / L::NST + 1) * WARPS - 1 && j + L::NST < t1) fill(u + L::NST);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      atomicOr(&g_err_kv8_attn, ERRBIT_TIMEOUT);
      *failed = 1;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_sum[n][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) {
          ml[warp * RT + 8 * n + 2 * t + c] = m_used[n][c];
          ml[(WARPS + warp) * RT + 8 * n + 2 * t + c] = l;
        }
      }
  }
  // ------------------------------------------------------------------ merge of the warps
  // (after this barrier every stage has been consumed: the stages' memory is free)
  __syncthreads();
  if (*failed) {   // unless a wait gave up: then the copies in flight get as long again
    if (tid == 0)
      for (int k = *issued > L::NST ? (int)*issued - L::NST : 0; k < (int)*issued; ++k)
        tc::mbar_wait(&full[k % L::NST], (k / L::NST) & 1);
    __syncthreads();
  }
  float* om = reinterpret_cast<float*>(base);    // [WARPS][RT][HD]
  {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * t + c;
        float mm = kNone, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, ml[w * RT + r]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) sum = fmaf(ml[(WARPS + w) * RT + r], tc::ex2_approx(ml[w * RT + r] - mm), sum);
        const float a = tc::ex2_approx(m_used[n][c] - mm);
        if (warp == 0 && g == 0) {
          cm[r] = mm;
          cm[RT + r] = sum;
        }
        // this thread's channels of row r: (HD/8) g + 0 .. HD/8 - 1, rotated by the row's pair so
        // that the four t of a store meet different banks
        float* dst = om + (warp * RT + r) * HD;
#pragma unroll
        for (int i = 0; i < KS; i += 2) {
          const int w4 = (HD / 32) * g + i / 2;               // 16-byte word of the row
          *reinterpret_cast<float4*>(dst + ((w4 + 2 * r) & (HD / 4 - 1)) * 4) =
              make_float4(O[i][n][c] * a, O[i][n][c + 2] * a, O[i + 1][n][c] * a, O[i + 1][n][c + 2] * a);
        }
      }
  }
  __syncthreads();
  for (int i = tid; i < RT * HD / 4; i += THREADS) {
    float4 x = reinterpret_cast<float4*>(om)[i];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      const float4 y = reinterpret_cast<float4*>(om)[w * (RT * HD / 4) + i];
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    reinterpret_cast<float4*>(om)[i] = x;
  }
  // ------------------------------------------------------------------ merge of the cluster
  if (n_split > 1)
    tc::cluster_sync();
  else
    __syncthreads();
  const uint32_t cm_a = tc::smem_u32(cm), om_a = tc::smem_u32(om);
  float* pf = ml;                          // [n_split][RT] factor of each CTA's part (the warps' figures are spent)
  if (tid < RT) {
    float mm = kNone, sum = 0.f;
    for (int c = 0; c < n_split; ++c) mm = fmaxf(mm, ld_cluster(tc::mapa_shared(cm_a + 4 * tid, c)));
    for (int c = 0; c < n_split; ++c) {
      const float f = tc::ex2_approx(ld_cluster(tc::mapa_shared(cm_a + 4 * tid, c)) - mm);
      pf[c * RT + tid] = f;
      sum = fmaf(ld_cluster(tc::mapa_shared(cm_a + 4 * (RT + tid), c)), f, sum);
    }
    fm[tid] = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);   // a row that sees nothing is 0, a NaN stays one
    // log2 of sum_i 2^z_i: the weights carry 2^(bias - m); a row that sees nothing weighs nothing
    fm[RT + tid] = sum == 0.f ? INFINITY : mm - kPBias + log2f(sum);
    if (p.lse && rank == 0 && tid < nrow) p.lse[head * R + row0 + tid] = fm[RT + tid];
  }
  __syncthreads();
  {
    // CTA `rank` writes an equal share of the tile's output
    const int n4 = nrow * (HD / 4), per = (n4 + n_split - 1) / n_split;
    T* out = static_cast<T*>(p.out);
    for (int i = rank * per + tid; i < min(n4, (rank + 1) * per); i += THREADS) {
      const int r = i / (HD / 4), w4 = i - r * (HD / 4);
      const uint32_t at = om_a + 16 * (r * (HD / 4) + ((w4 + 2 * r) & (HD / 4 - 1)));
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < n_split; ++c) {
        const float f = pf[c * RT + r];
        const float4 v = tc::ld_cluster4(tc::mapa_shared(at, c));
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
        o[2] = fmaf(v.z, f, o[2]);
        o[3] = fmaf(v.w, f, o[3]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] *= fm[r];
      const int rr = row0 + r, j = rr / p.G;
      st4(out + (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (rr - j * p.G)) * HD + 4 * w4, o);
    }
  }
  // ------------------------------------------------------------------ the keys' weights
  // (written back by the CTA that scored them: its own z, read after the barriers above)
  if (p.weights) {
    float* wr = p.weights + head * cap;
    const float* z = p.z + head * R * cap;
    const int64_t k1 = (int64_t)t1 * L::KT < nk ? (int64_t)t1 * L::KT : nk;
    for (int64_t key = (int64_t)t0 * L::KT + tid; key < k1; key += THREADS) {
      float sum = 0.f;
      for (int r = 0; r < nrow; ++r)       // an unseen key's z is -inf
        sum += tc::ex2_approx(z[r * cap + key] - fm[RT + r]);
      wr[key] += sum;
    }
  }
  if (n_split > 1) tc::cluster_sync();     // the peers may still be reading this CTA's part
}

// The weights of more query rows than one tile holds: with log2 of every row's sum known, each
// warp takes 16 keys (their codes stay in registers as matrix operands) and walks all query
// rows that can see them.  The sum over rows runs in a fixed order.
constexpr int ROWS = 16;
constexpr int WK_WARPS = 8;
template <int HD, typename T>
__global__ void __launch_bounds__(32 * WK_WARPS) k_kv8_weights(const Kv8Attn p) {
  pdl_wait();
  pdl_trigger();
  constexpr int NS = sizeof(T) == 4 ? 2 : 1;
  constexpr int KS = HD / 16;
  // one tile of 16 query rows as fp16 fragments, shared by the CTA's warps
  __shared__ uint4 sq[NS * KS * 32];
  __shared__ float s_f[ROWS], s_l[ROWS];
  __shared__ int s_last[ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, s = blockIdx.z;
  const int64_t cap = p.c.capacity, head = (int64_t)s * p.Hkv + h;
  const int64_t key0 = ((int64_t)blockIdx.x * WK_WARPS + warp) * 16;
  const int64_t cta_key0 = (int64_t)blockIdx.x * WK_WARPS * 16;
  const int R = p.n_q * p.G;
  const bool live = key0 < cap;
  uint32_t kb[2][KS][2];
  float ksg = 1.0f;
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t w = 0;
      if (live)
        w = *reinterpret_cast<const uint32_t*>(p.c.k_codes + (head * cap + key0 + n * 8 + g) * HD + t * (HD / 4) + 4 * ks);
      codes_to_h2(w, kb[n][ks][0], kb[n][ks][1]);
    }
  if (live) ksg = fmaxf(p.c.k_scale[head * (cap >> p.lg) + (key0 >> p.lg)], kKv8MinScale);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};    // keys 2t, 2t + 1 of both groups of 8
  bool any = false;
  for (int row0 = 0; row0 < R; row0 += ROWS) {
    const int nrow = min(ROWS, R - row0);
    __syncthreads();
    if (tid < ROWS) {
      int l = -1;
      if (tid < nrow) {
        l = p.last[(int64_t)s * p.n_q + (row0 + tid) / p.G];
        if (l < -1 || l >= cap) l = -1;    // reported by the attention kernel
      }
      s_last[tid] = l;
      s_l[tid] = tid < nrow ? p.lse[head * R + row0 + tid] : INFINITY;
    }
    __syncthreads();
    int mx = -1;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) mx = max(mx, s_last[i]);
    if (mx < cta_key0) continue;           // no row of the tile sees any key of the CTA
    if (warp == 0) {
      const T* q = static_cast<const T*>(p.q);
      float f[2][KS][4], amax[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool on = g + 8 * i < nrow;
        const int r = row0 + g + 8 * i, j = on ? r / p.G : 0;
        const T* qr = q + (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (on ? r - j * p.G : 0)) * HD + t * (HD / 4);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          load4(qr + 4 * ks, on, f[i][ks]);
#pragma unroll
          for (int c = 0; c < 4; ++c) amax[i] = fmaxf(amax[i], fabsf(f[i][ks][c]));
        }
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 1));
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 2));
        int e = amax[i] > 0.f ? ilogbf(amax[i]) : 0;
        e = e < -120 ? -120 : (e > 120 ? 120 : e);
        const float down = ldexpf(1.0f, -e);
        if (t == 0) s_f[g + 8 * i] = ldexpf(p.scale_log2, e);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int c = 0; c < 4; ++c) f[i][ks][c] *= down;
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 a = make_uint4(pack_h2(f[0][ks][0], f[0][ks][1]), pack_h2(f[1][ks][0], f[1][ks][1]),
                                   pack_h2(f[0][ks][2], f[0][ks][3]), pack_h2(f[1][ks][2], f[1][ks][3]));
        sq[ks * 32 + lane] = a;
        if constexpr (NS == 2)
          sq[(KS + ks) * 32 + lane] = make_uint4(rest_h2(f[0][ks][0], f[0][ks][1], a.x), rest_h2(f[1][ks][0], f[1][ks][1], a.y),
                                                 rest_h2(f[0][ks][2], f[0][ks][3], a.z), rest_h2(f[1][ks][2], f[1][ks][3], a.w));
      }
    }
    __syncthreads();
    if (!live || mx < key0) continue;
    any = true;
    float S[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[n][c] = 0.f;
#pragma unroll
    for (int part = 0; part < NS; ++part)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 a4 = sq[(part * KS + ks) * 32 + lane];
        const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int n = 0; n < 2; ++n) mma_f16(S[n], a, kb[n][ks][0], kb[n][ks][1]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = s_f[g + 8 * i] * ksg, l = s_l[g + 8 * i];
      const int lst = s_last[g + 8 * i];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if ((int)key0 + n * 8 + 2 * t + c <= lst) sum[2 * n + c] += tc::ex2_approx(fmaf(S[n][2 * i + c], f, -l));
    }
  }
  if (!any) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
  if (g == 0) {
    float* w = p.weights + head * cap + key0;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (sum[2 * n + c] != 0.f) w[n * 8 + 2 * t + c] += sum[2 * n + c];
  }
}

// shared-memory limits set per device and kernel, guarded for calls from several host threads
std::mutex g_kv8_mu;
uint32_t g_kv8_attr[64];
int g_kv8_sms[64];

template <int HD, int NT, typename T>
cudaError_t prepare_attn(int dev) {
  constexpr int h = HD == 32 ? 0 : HD == 64 ? 1 : HD == 128 ? 2 : 3;
  constexpr uint32_t bit = 1u << (h + (sizeof(T) == 4 ? 4 : 0) + (NT == 2 ? 8 : 0));
  std::lock_guard<std::mutex> g(g_kv8_mu);
  if (dev >= 0 && dev < 64 && (g_kv8_attr[dev] & bit)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn<HD, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       SmemOf<HD, NT, T>::BYTES);
  if (e == cudaSuccess && dev >= 0 && dev < 64) g_kv8_attr[dev] |= bit;
  return e;
}

int device_sms(int dev) {
  std::lock_guard<std::mutex> g(g_kv8_mu);
  if (dev >= 0 && dev < 64 && g_kv8_sms[dev]) return g_kv8_sms[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();   // clears the error of the call just made (nothing is cached)
    return 148;
  }
  if (dev >= 0 && dev < 64) g_kv8_sms[dev] = n;
  return n;
}

// rows of a tile of k_kv8_attn: 8 where they suffice (and at head_dim 256, for the registers)
int tile_rows(int hd, int64_t R) { return hd == 256 || R <= 8 ? 8 : 16; }

template <int HD, int NT, typename T>
cudaError_t launch_attn_n(const Kv8Attn& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = prepare_attn<HD, NT, T>(dev)) != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)p.n_q * p.G + 8 * NT - 1) / (8 * NT);
  const int64_t units = tiles * p.Hkv * p.c.n_seq, kt = (p.c.capacity + Lay<HD>::KT - 1) / Lay<HD>::KT;
  const int64_t want = 2 * (int64_t)device_sms(dev);
  int ns = 1;
  while (ns < MAX_SPLIT && units * ns < want && 2 * ns <= kt) ns *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ns), p.Hkv, p.c.n_seq);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SmemOf<HD, NT, T>::BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ns;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_kv8_attn<HD, NT, T>, p, ns);
}

template <int HD, typename T>
cudaError_t launch_attn_t(const Kv8Attn& p, cudaStream_t s) {
  if constexpr (HD < 256)
    if (tile_rows(HD, (int64_t)p.n_q * p.G) == 16) return launch_attn_n<HD, 2, T>(p, s);
  return launch_attn_n<HD, 1, T>(p, s);
}

template <int HD, typename T>
cudaError_t launch_weights_t(const Kv8Attn& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.c.capacity + 16 * WK_WARPS - 1) / (16 * WK_WARPS)), p.Hkv, p.c.n_seq);
  return launch_k(k_kv8_weights<HD, T>, grid, dim3(32 * WK_WARPS), 0, s, p);
}

}  // namespace

void reset_kv8_attn_caches() {
  std::lock_guard<std::mutex> g(g_kv8_mu);
  for (int i = 0; i < 64; ++i) {
    g_kv8_attr[i] = 0;
    g_kv8_sms[i] = 0;
  }
}

bool kv8_attn_supported(int hd) { return hd == 32 || hd == 64 || hd == 128 || hd == 256; }

// whether the weights take a launch of their own: the rows do not fit in one tile
bool kv8_attn_weights_apart(int hd, int G, int n_q) {
  const int64_t R = (int64_t)n_q * G;
  return R > tile_rows(hd, R);
}

// scratch for the weights: the scores of the rows, or log2 of every row's sum
size_t kv8_attn_ws_bytes(int n_seq, int Hkv, int G, int n_q, int64_t cap, int hd, bool weights) {
  if (!weights) return 0;
  const size_t R = (size_t)n_q * G;
  return (size_t)n_seq * Hkv * 4 * R * (kv8_attn_weights_apart(hd, G, n_q) ? 1 : (size_t)cap);
}

static Kv8Attn make_params(const void* q, const int32_t* last, int n_q, const cb_kv8_cache& c, int H, int Hkv, int hd,
                           void* out, float* weights, void* ws) {
  Kv8Attn p{};
  p.q = q;
  p.last = last;
  p.out = out;
  p.c = c;
  p.n_q = n_q;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.lg = 31 - __builtin_clz((unsigned)c.block);
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)hd);
  if (weights) {
    if (kv8_attn_weights_apart(hd, p.G, n_q)) {
      p.lse = static_cast<float*>(ws);
    } else {
      p.z = static_cast<float*>(ws);
      p.weights = weights;
    }
  }
  return p;
}

#define CB_KV8_DISPATCH(fn)                                                      \
  switch (hd) {                                                                  \
    case 32: return dt == DT_BF16 ? fn<32, bf16>(p, s) : fn<32, float>(p, s);    \
    case 64: return dt == DT_BF16 ? fn<64, bf16>(p, s) : fn<64, float>(p, s);    \
    case 128: return dt == DT_BF16 ? fn<128, bf16>(p, s) : fn<128, float>(p, s); \
    case 256: return dt == DT_BF16 ? fn<256, bf16>(p, s) : fn<256, float>(p, s); \
    default: return cudaErrorInvalidValue;                                       \
  }

cudaError_t launch_kv8_attn(int dt, const void* q, const int32_t* last, int n_q, const cb_kv8_cache& c, int H, int Hkv,
                            int hd, void* out, float* weights, void* ws, cudaStream_t s) {
  const Kv8Attn p = make_params(q, last, n_q, c, H, Hkv, hd, out, weights, ws);
  CB_KV8_DISPATCH(launch_attn_t)
}

cudaError_t launch_kv8_weights(int dt, const void* q, const int32_t* last, int n_q, const cb_kv8_cache& c, int H,
                               int Hkv, int hd, float* weights, void* ws, cudaStream_t s) {
  Kv8Attn p = make_params(q, last, n_q, c, H, Hkv, hd, nullptr, weights, ws);
  p.weights = weights;
  CB_KV8_DISPATCH(launch_weights_t)
}

}  // namespace cb
