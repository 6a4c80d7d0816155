// Attention over the 8-bit block-scaled KV cache (cb_kv8.cu), for a few query rows per KV head
// (single tokens) and, in tiles of 16 rows, for any number.
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

constexpr int ROWS = 16;             // query rows per tile: the M of mma.m16n8k16
constexpr int WARPS = 4;             // consumer warps; one more warp produces
constexpr int THREADS = 32 * (WARPS + 1);
constexpr float kPBias = 8.0f;       // 2^(t - m) is held up to 2^8 ...
constexpr float kLazy = 6.0f;        // ... and up to 2^14 before m is raised: fp16 ends at 2^16

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

struct Kv8Attn {
  const void* q;
  const int32_t* last;      // [n_seq, n_q]
  void* out;
  float* z;                 // [n_seq * Hkv, ROWS, capacity] scores z_i for the weights, or null
  float* lse;               // [n_seq, Hkv, n_q * G] log2 of a row's sum, or null
  float* weights;           // [n_seq, Hkv, capacity] (with z), or null
  cb_kv8_cache c;
  int n_q, H, Hkv, G, lg;
  float scale_log2;         // log2(e) / sqrt(hd)
};

// a stage holds KT keys: 16 or 32 per warp, so that a stage is at least 8 KB of codes
template <int HD>
struct Lay {
  static constexpr int KW = HD <= 64 ? 2 : 1;                      // groups of 16 keys per warp and stage
  static constexpr int KT = 16 * WARPS * KW;
  static constexpr int HALF = KT * HD;                             // K (or V) codes of a stage
  static constexpr int NST = (98304 / (2 * HALF)) > 8 ? 8 : 98304 / (2 * HALF);
  static constexpr int NG = KT / 16;
  static constexpr int OFF_SC = NST * 2 * HALF;                    // [NST][3][NG] ks, log2 vs, 1/vs
  static constexpr int OFF_ML = OFF_SC + NST * 3 * NG * 4;         // row max and sum per warp, per CTA, ...
  static constexpr int N_ML = 2 * WARPS * ROWS + 4 * ROWS;
  static constexpr int OFF_LAST = OFF_ML + N_ML * 4;               // [ROWS]
  static constexpr int OFF_BAR = OFF_LAST + ROWS * 4 + 16;
  static constexpr int OFF_Q = OFF_BAR + 2 * NST * 8;              // fp16 q in fragment order (when not in registers)
  static_assert(OFF_BAR % 8 == 0 && OFF_Q % 16 == 0, "barriers or q misaligned");
  static_assert(WARPS * ROWS * HD * 4 <= OFF_SC, "the merge buffer exceeds the stages");
};
template <int HD, typename T>
constexpr bool q_in_smem() {
  return HD == 256 || sizeof(T) == 4;
}
template <int HD, typename T>
constexpr int smem_bytes() {
  return Lay<HD>::OFF_Q + (q_in_smem<HD, T>() ? (sizeof(T) == 4 ? 2 : 1) * ROWS * HD * 2 : 0) + 128;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, bool on, float* f) {
  if (on) {
    ld4(p, f);
  } else {
    f[0] = f[1] = f[2] = f[3] = 0.f;
  }
}

// One cluster of gridDim-x-fastest CTAs per (16 query rows, KV head, sequence); its CTAs take
// consecutive runs of the visible keys and are merged through distributed shared memory.
template <int HD, typename T>
__global__ void __launch_bounds__(THREADS, HD == 256 ? 1 : 2) k_kv8_attn(const Kv8Attn p, int n_split) {
  pdl_wait();
  pdl_trigger();
  using L = Lay<HD>;
  constexpr int NS = sizeof(T) == 4 ? 2 : 1;     // fp16 parts of q and of the weights
  constexpr bool QS = q_in_smem<HD, T>();
  constexpr int KS = HD / 16;                    // k steps of a score, and pairs of output tiles
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((128 - (tc::smem_u32(smem_raw) & 127)) & 127);
  float* ssc = reinterpret_cast<float*>(base + L::OFF_SC);
  float* ml = reinterpret_cast<float*>(base + L::OFF_ML);
  int* slast = reinterpret_cast<int*>(base + L::OFF_LAST);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + L::OFF_BAR);
  uint64_t* empty = full + L::NST;
  uint32_t* sq = reinterpret_cast<uint32_t*>(base + L::OFF_Q);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % n_split, rt = blockIdx.x / n_split, h = blockIdx.y, s = blockIdx.z;
  const int R = p.n_q * p.G, row0 = rt * ROWS, nrow = min(ROWS, R - row0);
  const int64_t cap = p.c.capacity, head = (int64_t)s * p.Hkv + h;

  if (tid < ROWS) {
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
      tc::mbar_init(&empty[i], WARPS);
    }
    tc::fence_mbar_init();
  }
  __syncthreads();
  int mx = -1, mn = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    mx = max(mx, slast[i]);
    if (i < nrow) mn = min(mn, slast[i]);
  }
  const int64_t nk = (int64_t)mx + 1;                        // keys some row sees
  const int tiles = (int)((nk + L::KT - 1) / L::KT);
  const int t0 = (int)((int64_t)tiles * rank / n_split), t1 = (int)((int64_t)tiles * (rank + 1) / n_split);
  const int64_t nblk = cap >> p.lg;

  float O[2 * KS][4];
  float m_used[2] = {-INFINITY, -INFINITY}, l_sum[2] = {0.f, 0.f};
  bool ok = true;

  if (warp == WARPS) {
    // ------------------------------------------------------------------ producer warp
    const int8_t* kc = p.c.k_codes + head * cap * HD;
    const int8_t* vc = p.c.v_codes + head * cap * HD;
    const float* ksc = p.c.k_scale + head * nblk;
    const float* vsc = p.c.v_scale + head * nblk;
    // lane l < NG: group l's K scale, NG <= l < 2 NG: V's; a group past the visible keys gets
    // scale 1 (its block may never have been written)
    auto scale_of = [&](int j) -> float {
      const int64_t key = (int64_t)j * L::KT + 16 * (lane % L::NG);
      if (lane >= 2 * L::NG || j >= t1 || key >= nk) return 1.0f;
      return (lane < L::NG ? ksc : vsc)[key >> p.lg];
    };
    float sc = scale_of(t0);
    int u = 0;
    for (; u < t1 - t0; ++u) {
      const int j = t0 + u, st = u % L::NST;
      const float nxt = scale_of(j + 1);
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[st], ((u / L::NST) & 1) ^ 1));
      if (!ok) break;
      float* dst = ssc + st * 3 * L::NG;
      if (lane < L::NG) {
        dst[lane] = fmaxf(sc, kKv8MinScale);
      } else if (lane < 2 * L::NG) {
        const float v = fmaxf(sc, kKv8MinScale);
        dst[lane] = log2f(v);
        dst[lane + L::NG] = 1.0f / v;
      }
      sc = nxt;
      __syncwarp();
      if (lane == 0) {
        const int64_t k0 = (int64_t)j * L::KT;
        const uint32_t bytes = (uint32_t)(cap - k0 < L::KT ? cap - k0 : L::KT) * HD;
        tc::mbar_expect_tx(&full[st], 2 * bytes);
        bulk_load(base + st * 2 * L::HALF, kc + k0 * HD, bytes, &full[st]);
        bulk_load(base + st * 2 * L::HALF + L::HALF, vc + k0 * HD, bytes, &full[st]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(&g_err_kv8_attn, ERRBIT_TIMEOUT);
    // no copy is in flight when the CTA goes on, whoever gave up on what
    for (int k = u > L::NST ? u - L::NST : 0; k < u; ++k) tc::mbar_wait(&full[k % L::NST], (k / L::NST) & 1);
  } else {
    // ------------------------------------------------------------------ consumer warps
    const bool upper = nrow > 8;                              // rows 8..15 exist
    // q rows g and g + 8: channels [t HD/4, (t + 1) HD/4), 4 per k step (the order of the
    // channels inside a sum is free; K is read with the same one)
    float rf[2];                                              // score factor of the rows
    uint32_t qa[QS ? 1 : KS][4];
    {
      const T* q = static_cast<const T*>(p.q);
      const T* qr[2];
      bool on[2];
      float amax[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + g + 8 * i;
        on[i] = g + 8 * i < nrow;
        const int j = on[i] ? r / p.G : 0;
        qr[i] = q + (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (on[i] ? r - j * p.G : 0)) * HD + t * (HD / 4);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          float f[4];
          load4(qr[i] + 4 * ks, on[i], f);
          amax[i] = fmaxf(amax[i], fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
        }
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 1));
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 2));
      }
      float down[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // 2^e <= amax < 2^(e + 1); both powers stay normal
        int e = amax[i] > 0.f ? ilogbf(amax[i]) : 0;
        e = e < -120 ? -120 : (e > 120 ? 120 : e);
        down[i] = ldexpf(1.0f, -e);
        rf[i] = ldexpf(p.scale_log2, e);
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        float f0[4], f1[4];
        load4(qr[0] + 4 * ks, on[0], f0);
        load4(qr[1] + 4 * ks, on[1], f1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f0[i] *= down[0];
          f1[i] *= down[1];
        }
        uint32_t a[4] = {pack_h2(f0[0], f0[1]), pack_h2(f1[0], f1[1]), pack_h2(f0[2], f0[3]), pack_h2(f1[2], f1[3])};
        if constexpr (QS) {
          if (warp == 0) {
            *reinterpret_cast<uint4*>(sq + (ks * 32 + lane) * 4) = make_uint4(a[0], a[1], a[2], a[3]);
            if constexpr (NS == 2)
              *reinterpret_cast<uint4*>(sq + ((KS + ks) * 32 + lane) * 4) =
                  make_uint4(rest_h2(f0[0], f0[1], a[0]), rest_h2(f1[0], f1[1], a[1]), rest_h2(f0[2], f0[3], a[2]),
                             rest_h2(f1[2], f1[3], a[3]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) qa[ks][i] = a[i];
        }
      }
      if constexpr (QS) asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
    }
    const int last0 = slast[g], last1 = slast[g + 8];
    float* zrow = p.z ? p.z + head * ROWS * cap : nullptr;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) O[i][c] = 0.f;

    for (int j = t0; j < t1; ++j) {
      const int u = j - t0, st = u % L::NST;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[st], (u / L::NST) & 1));
      if (!ok) break;
      const uint8_t* sk = base + st * 2 * L::HALF;
      const float* sc = ssc + st * 3 * L::NG;
#pragma unroll 1
      for (int w = 0; w < L::KW; ++w) {
        const int grp = warp * L::KW + w;
        const int64_t key0 = (int64_t)j * L::KT + grp * 16;
        if (key0 >= nk) break;
        // ---- scores of 16 keys
        float S[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int c = 0; c < 4; ++c) S[n][c] = 0.f;
          const uint8_t* kr = sk + (grp * 16 + n * 8 + g) * HD + t * (HD / 4);
          uint32_t kw[KS];
          if constexpr (HD >= 64) {
#pragma unroll
            for (int i = 0; i < KS / 4; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(kr + 16 * i);
              kw[4 * i] = v.x;
              kw[4 * i + 1] = v.y;
              kw[4 * i + 2] = v.z;
              kw[4 * i + 3] = v.w;
            }
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kr);
            kw[0] = v.x;
            kw[1] = v.y;
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t b0, b1;
            codes_to_h2(kw[ks], b0, b1);
            if constexpr (QS) {
#pragma unroll
              for (int part = 0; part < NS; ++part) {
                const uint4 a4 = *reinterpret_cast<const uint4*>(sq + ((part * KS + ks) * 32 + lane) * 4);
                const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w};
                mma_f16(S[n], a, b0, b1);
              }
            } else {
              mma_f16(S[n], qa[ks], b0, b1);
            }
          }
        }
        // ---- weights of the 16 keys, rows g (half 0) and g + 8 (half 1)
        const float ksg = sc[grp], lvs = sc[L::NG + grp], ivs = sc[2 * L::NG + grp];
        const bool whole = key0 + 15 <= mn;                   // every row sees every key
        float mt[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !upper) {
            mt[1] = -INFINITY;
            break;
          }
          const float f = rf[i] * ksg;
          const int lst = i ? last1 : last0;
          float mm = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int key = (int)key0 + n * 8 + 2 * t + c;
              float z = S[n][2 * i + c] * f;
              if (!whole && key > lst) z = -INFINITY;
              S[n][2 * i + c] = z;
              mm = fmaxf(mm, z);
            }
          if (zrow && g + 8 * i < nrow) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
              *reinterpret_cast<float2*>(zrow + (int64_t)(g + 8 * i) * cap + key0 + n * 8 + 2 * t) =
                  make_float2(S[n][2 * i], S[n][2 * i + 1]);
          }
          mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
          mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
          mt[i] = mm + lvs;
        }
        // m is raised when a weight would leave fp16's range (and at the row's first key)
        const bool up0 = mt[0] > m_used[0] + kLazy, up1 = mt[1] > m_used[1] + kLazy;
        if (__any_sync(0xffffffffu, up0 || up1)) {
          const float a0 = up0 ? tc::ex2_approx(m_used[0] - mt[0]) : 1.0f;
          const float a1 = up1 ? tc::ex2_approx(m_used[1] - mt[1]) : 1.0f;
          if (up0) m_used[0] = mt[0];
          if (up1) m_used[1] = mt[1];
          l_sum[0] *= a0;
          l_sum[1] *= a1;
#pragma unroll
          for (int i = 0; i < 2 * KS; ++i) {
            O[i][0] *= a0;
            O[i][1] *= a0;
            O[i][2] *= a1;
            O[i][3] *= a1;
          }
        }
        uint32_t pa[NS][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !upper) {
#pragma unroll
            for (int part = 0; part < NS; ++part) pa[part][1] = pa[part][3] = 0u;
            break;
          }
          // a row that has seen nothing yet keeps weights of 0
          const float add = lvs - (m_used[i] == -INFINITY ? 0.f : m_used[i]) + kPBias;
          float e[2][2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            e[n][0] = tc::ex2_approx(S[n][2 * i] + add);
            e[n][1] = tc::ex2_approx(S[n][2 * i + 1] + add);
            pa[0][2 * n + i] = pack_h2(e[n][0], e[n][1]);
            if constexpr (NS == 2) pa[NS - 1][2 * n + i] = rest_h2(e[n][0], e[n][1], pa[0][2 * n + i]);
          }
          l_sum[i] = fmaf((e[0][0] + e[0][1]) + (e[1][0] + e[1][1]), ivs, l_sum[i]);
        }
        // ---- O += P V: this thread's V rows are keys 2t, 2t+1, 2t+8, 2t+9; column g of output
        // tile n stands for channel (HD/8) g + n
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
              v[r][0] = x.x;
              v[r][1] = x.y;
              v[r][2] = x.z;
              v[r][3] = x.w;
            } else if constexpr (VC == 8) {
              const uint2 x = *reinterpret_cast<const uint2*>(a);
              v[r][0] = x.x;
              v[r][1] = x.y;
            } else {
              v[r][0] = *reinterpret_cast<const uint32_t*>(a);
            }
          }
#pragma unroll
          for (int c = 0; c < VC / 4; ++c) {
            const uint32_t b0[4] = {codes_pair<0>(v[0][c], v[1][c]), codes_pair<1>(v[0][c], v[1][c]),
                                    codes_pair<2>(v[0][c], v[1][c]), codes_pair<3>(v[0][c], v[1][c])};
            const uint32_t b1[4] = {codes_pair<0>(v[2][c], v[3][c]), codes_pair<1>(v[2][c], v[3][c]),
                                    codes_pair<2>(v[2][c], v[3][c]), codes_pair<3>(v[2][c], v[3][c])};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int part = 0; part < NS; ++part) mma_f16(O[c0 + 4 * c + q], pa[part], b0[q], b1[q]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[st]);
    }
    if (!ok && lane == 0) atomicOr(&g_err_kv8_attn, ERRBIT_TIMEOUT);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l_sum[i] += __shfl_xor_sync(0xffffffffu, l_sum[i], 1);
      l_sum[i] += __shfl_xor_sync(0xffffffffu, l_sum[i], 2);
      if (t == 0) {
        ml[warp * ROWS + g + 8 * i] = m_used[i];
        ml[(WARPS + warp) * ROWS + g + 8 * i] = l_sum[i];
      }
    }
  }
  // ------------------------------------------------------------------ merge of the warps
  // (after this barrier every stage has been consumed: the stages' memory is free)
  __syncthreads();
  float* cm = ml + 2 * WARPS * ROWS;       // [ROWS] CTA max, then [ROWS] CTA sum
  float* fm = cm + 2 * ROWS;               // [ROWS] 1 / sum over the cluster, [ROWS] log2 of it
  float* om = reinterpret_cast<float*>(base);
  if (warp < WARPS) {
    float a[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w * ROWS + r]);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float mw = ml[w * ROWS + r];
        if (mw > -INFINITY) sum = fmaf(ml[(WARPS + w) * ROWS + r], tc::ex2_approx(mw - M), sum);
      }
      a[i] = m_used[i] > -INFINITY ? tc::ex2_approx(m_used[i] - M) : 0.f;
      if (warp == 0 && t == 0) {
        cm[r] = M;
        cm[ROWS + r] = sum;
      }
    }
    // this thread's columns: channels (HD/8)(2t + c) + n
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* dst = om + (warp * ROWS + g + 8 * i) * HD + (HD / 8) * (2 * t + c);
#pragma unroll
        for (int n = 0; n < HD / 8; n += 4)
          *reinterpret_cast<float4*>(dst + n) =
              make_float4(O[n][2 * i + c] * a[i], O[n + 1][2 * i + c] * a[i], O[n + 2][2 * i + c] * a[i],
                          O[n + 3][2 * i + c] * a[i]);
      }
  }
  __syncthreads();
  for (int i = tid; i < ROWS * HD / 4; i += THREADS) {
    float4 x = reinterpret_cast<float4*>(om)[i];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      const float4 y = reinterpret_cast<float4*>(om)[w * (ROWS * HD / 4) + i];
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
  float* pf = ml;                          // [n_split][ROWS] factor of each CTA's part (the warps' figures are spent)
  if (tid < ROWS) {
    float M = -INFINITY, sum = 0.f;
    for (int c = 0; c < n_split; ++c) M = fmaxf(M, ld_cluster(tc::mapa_shared(cm_a + 4 * tid, c)));
    for (int c = 0; c < n_split; ++c) {
      const float mc = ld_cluster(tc::mapa_shared(cm_a + 4 * tid, c));
      const float f = mc > -INFINITY ? tc::ex2_approx(mc - M) : 0.f;
      pf[c * ROWS + tid] = f;
      sum = fmaf(ld_cluster(tc::mapa_shared(cm_a + 4 * (ROWS + tid), c)), f, sum);
    }
    fm[tid] = sum > 0.f ? 1.0f / sum : 0.f;
    // log2 of sum_i 2^z_i: the weights carry 2^(m - bias); a row that sees nothing weighs nothing
    fm[ROWS + tid] = sum > 0.f ? M - kPBias + log2f(sum) : INFINITY;
    if (p.lse && rank == 0 && tid < nrow) p.lse[head * R + row0 + tid] = fm[ROWS + tid];
  }
  __syncthreads();
  {
    // CTA `rank` writes an equal share of the tile's output
    constexpr int N4 = ROWS * HD / 4;
    const int per = (N4 + n_split - 1) / n_split;
    T* out = static_cast<T*>(p.out);
    for (int i = rank * per + tid; i < min(N4, (rank + 1) * per); i += THREADS) {
      const int r = i / (HD / 4), d = (i - r * (HD / 4)) * 4;
      if (r >= nrow) break;
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < n_split; ++c) {
        const float f = pf[c * ROWS + r];
        if (f == 0.f) continue;            // also a CTA without visible keys
        const float4 v = tc::ld_cluster4(tc::mapa_shared(om_a + 16 * i, c));
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
        o[2] = fmaf(v.z, f, o[2]);
        o[3] = fmaf(v.w, f, o[3]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] *= fm[r];
      const int rr = row0 + r, j = rr / p.G;
      st4(out + (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (rr - j * p.G)) * HD + d, o);
    }
  }
  // ------------------------------------------------------------------ the keys' weights
  // (written back by the CTA that scored them: its own z, read after the barriers above)
  if (p.weights) {
    float* wr = p.weights + head * cap;
    const float* z = p.z + head * ROWS * cap;
    const int64_t k1 = (int64_t)t1 * L::KT < nk ? (int64_t)t1 * L::KT : nk;
    for (int64_t key = (int64_t)t0 * L::KT + tid; key < k1; key += THREADS) {
      float sum = 0.f;
      for (int r = 0; r < nrow; ++r)       // an unseen key's z is -inf
        sum += tc::ex2_approx(z[r * cap + key] - fm[ROWS + r]);
      wr[key] += sum;
    }
  }
  if (n_split > 1) tc::cluster_sync();     // the peers may still be reading this CTA's part
}

// The weights of more than 16 query rows per KV head: with log2 of every row's sum known, each
// warp takes 16 keys (their codes stay in registers as matrix operands) and walks all query
// rows that can see them.  The sum over rows runs in a fixed order.
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

template <int HD, typename T>
cudaError_t prepare_attn(int dev) {
  constexpr uint32_t bit = 1u << ((HD == 32 ? 0 : HD == 64 ? 1 : HD == 128 ? 2 : 3) + (sizeof(T) == 4 ? 4 : 0));
  std::lock_guard<std::mutex> g(g_kv8_mu);
  if (dev >= 0 && dev < 64 && (g_kv8_attr[dev] & bit)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<HD, T>());
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

template <int HD, typename T>
cudaError_t launch_attn_t(const Kv8Attn& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = prepare_attn<HD, T>(dev)) != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)p.n_q * p.G + ROWS - 1) / ROWS;
  const int64_t units = tiles * p.Hkv * p.c.n_seq, kt = (p.c.capacity + Lay<HD>::KT - 1) / Lay<HD>::KT;
  const int64_t want = 2 * (int64_t)device_sms(dev);
  int ns = 1;
  while (ns < 8 && units * ns < want && 2 * ns <= kt) ns *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ns), p.Hkv, p.c.n_seq);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes<HD, T>();
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
  return cudaLaunchKernelEx(&cfg, k_kv8_attn<HD, T>, p, ns);
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

// scratch for the weights: the scores of a 16-row tile, or log2 of every row's sum
size_t kv8_attn_ws_bytes(int n_seq, int Hkv, int G, int n_q, int64_t cap, bool weights) {
  if (!weights) return 0;
  const int64_t R = (int64_t)n_q * G;
  return (size_t)n_seq * Hkv * 4 * (size_t)(R <= ROWS ? ROWS * cap : R);
}

bool kv8_attn_weights_apart(int G, int n_q) { return (int64_t)n_q * G > ROWS; }

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
    if (kv8_attn_weights_apart(p.G, n_q)) {
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
