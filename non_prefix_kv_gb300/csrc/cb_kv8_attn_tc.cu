// Attention of many query rows over the 8-bit block-scaled KV cache on the tensor cores
// (head_dim 64 or 128), and the attention weight each cache row receives from them.
//
// The mathematics is cb_kv8_attn.cu's: the codes enter the matrix instructions exactly, K's
// scale multiplies a score, V's scale sits in the exponent (t = z + log2 vs) and leaves the
// row sum by a multiplication with 1 / vs.  Here
//   S_j = Q C_K,j^T    tcgen05.mma, bf16 x bf16 (an 8-bit code is exact in bf16), into TMEM
//   P_j = 2^(t - m)    softmax warps, fp16, back into TMEM
//   O  += P_j C_V,j    tcgen05.mma, fp16 x fp16, P from TMEM
// fp32 queries come, as there, as two fp16 parts of the row divided by a power of two, and P as two
// fp16 parts; the two products of each kind add up in the same accumulator.
// k_kv8_expand turns the codes into those two forms once per call, already in the swizzled
// order the tensor cores read, so that a tile is one bulk copy and no tensor map is needed:
// every key tile is read by n_q G / 128 CTAs, and converting it in each of them would cost
// more issue slots than the softmax itself (26 instructions per 16 codes, against one pass
// over 5 bytes per code).  With a single query tile each tile of the cache has one reader, which
// converts it itself (FUSED).
//
// Rows of one KV head are packed into tiles: row r of a tile is query r / G, head r % G, so
// a few queries of grouped heads fill a tile and a tile's rows share one narrow run of
// positions.  Small grids split the keys over a cluster of CTAs, merged through distributed
// shared memory.
#include <math.h>

#include <atomic>
#include <mutex>

#include "cb_kv8.cuh"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_kv8_tc;
static std::atomic<bool> g_used_kv8_tc{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_kv8_tc() { return g_used_kv8_tc ? take_word(g_err_kv8_tc) : 0u; }

namespace {

using tc::f2_add;
using tc::f2_fma;
using tc::f2_pack;
using tc::f2_unpack;
using tc::fmax3;

constexpr int BM = 128;              // query rows per tile
constexpr int BN = 128;              // keys per tile
constexpr int SLAB = 128 * 128;      // bytes of one [128 rows x 64 elements] swizzled slab
constexpr int NSOFT = 8;             // softmax warps: two groups of one per TMEM lane quarter
constexpr int ATTN_THREADS = 32 * NSOFT;           // of the attention kernel
constexpr int THREADS = 32 * (2 + NSOFT);          // of the weights kernel
constexpr uint32_t TMEM_COLS = 512;
constexpr int NG = BN / 16;          // scale groups of a key tile
// fp16 parts of q and of the weights (bf16 queries enter as they are)
template <typename T>
constexpr int parts() {
  return sizeof(T) == 4 ? 2 : 1;
}
// floats per query row that the weights' kernel reads
template <typename T>
constexpr int row_words() {
  return sizeof(T) == 4 ? 3 : 2;
}
constexpr float kPBias = 8.0f;       // as in cb_kv8_attn.cu: weights up to 2^8, 2^14 before m is raised
constexpr float kLazy = 6.0f;

struct Kv8Tc {
  const void* q;
  const int32_t* last;      // [n_seq, n_q]
  void* out;
  uint8_t* kx;              // [n_seq * Hkv, tiles] key tiles in shared-memory order: bf16 codes (fp32 queries: fp16)
  uint8_t* vx;              // the same of V: fp16 codes
  int32_t* seq_max;         // [n_seq] the last row any query of the sequence sees (for the weights)
  // for the weights (else null), per (sequence, KV head, query tile):
  uint8_t* qx;              // the tile's query rows in shared-memory order
  float* rows;              // [BM] log2 of each row's sum (+inf where there is none), [BM] last row it sees (int; -1: none),
                            // fp32: [BM] the row's power of two
  int32_t* tile_max;        // [n_seq, query tiles] the last row any query of the tile sees
  float* weights;           // [n_seq, Hkv, capacity]
  cb_kv8_cache c;
  int n_q, H, Hkv, G, lg, tiles, q_tiles;
  int qpt;                  // queries per tile: 128 / G
  int g_magic;              // ceil(2^16 / G): r / G = r g_magic >> 16 for r < 128
  float scale_log2;
};

__device__ __forceinline__ int last_of(const Kv8Tc& p, int s, int j) {
  const int l = p.last[(int64_t)s * p.n_q + j];
  return l < -1 || l >= p.c.capacity ? -1 : l;
}

// ---- codes to matrix operands -------------------------------------------------------------
// byte c of w as bf16 / fp16 pairs.  fp16: byte ^ 0x80 = c + 128, 0x6400 | u is 1024 + u.
// bf16 (7 mantissa bits): 0x4300 | (c & 127) is 128 + (c & 127); from it 128 is taken, or 256
// where the code is negative (0x4300 | (c & 128) is 128 or 256).
__device__ __forceinline__ uint32_t pair_f16(uint32_t u, uint32_t sel) {
  const uint32_t x = __byte_perm(u, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pair_bf16(uint32_t w, uint32_t sel) {
  const uint32_t x = __byte_perm(w, 0x43434343u, sel);
  const uint32_t a = x & 0xff7fff7fu, b = x & 0xff80ff80u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 32 bytes, the two halves exchanged if asked
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool swap) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = swap ? w[4 + i] : w[i];
    b[i] = swap ? w[i] : w[4 + i];
  }
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]),
               "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
               : "memory");
}

// One CTA per (key tile, KV head, sequence): 128 rows of K and V codes to bf16 / fp16 in
// 128-byte-swizzled slabs.  Tiles no query sees are skipped.  Bound by latency and L2 (34 MB of
// codes read, 67 MB written that the next kernel reads from L2): 15 us for 8 heads of 16384 rows,
// 19 us with 16-byte stores.  The loads come before it is known whether a query sees the tile, so a
// cache that is mostly empty is read whole: 832 rows of 32 heads over 1638 held rows 50 us in a cache
// for 16384 rows, 28 us in one for 1664 (at 16384 held rows 194 us).
template <int HD, typename T>
__global__ void __launch_bounds__(256) k_kv8_expand(const Kv8Tc p) {
  pdl_wait();
  pdl_trigger();
  const int tile = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int64_t head = (int64_t)s * p.Hkv + h, row0 = (int64_t)tile * BN;
  const int64_t src = (head * p.c.capacity + row0) * HD, dst = (head * p.tiles + tile) * (int64_t)(BN * HD * 2);
  constexpr int PER = HD / 16;             // pieces of 16 codes in a row
  constexpr int N = BN * PER / 256;        // pieces of a thread
  // all loads first: they and the look for a query that sees the tile share one latency
  uint4 k[N], v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int idx = i * 256 + threadIdx.x, row = idx / PER, piece = idx % PER;
    k[i] = v[i] = make_uint4(0, 0, 0, 0);
    if (row0 + row < p.c.capacity) {
      k[i] = *reinterpret_cast<const uint4*>(p.c.k_codes + src + row * HD + piece * 16);
      v[i] = *reinterpret_cast<const uint4*>(p.c.v_codes + src + row * HD + piece * 16);
    }
  }
  if (tile == 0 && h == 0) {               // the sequence's largest bound, for the kernels after this one
    int mx = -1;
    for (int j = threadIdx.x; j < p.n_q; j += 256) mx = max(mx, last_of(p, s, j));
    __shared__ int sm[8];
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = mx;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 0; w < 8; ++w) mx = max(mx, sm[w]);
      p.seq_max[s] = mx;
    }
  }
  // some query sees the tile's first key?  (the newest rows usually come last)
  bool need = false;
  for (int j = p.n_q - 1 - (int)threadIdx.x; !need; j -= 256) {
    need = __syncthreads_or(j >= 0 && last_of(p, s, j) >= tile * BN);
    if (__syncthreads_and(j < 256)) break;
  }
  if (!need) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int idx = i * 256 + threadIdx.x, row = idx / PER, piece = idx % PER;
    const uint32_t kw[4] = {k[i].x, k[i].y, k[i].z, k[i].w}, vw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    // 16 codes are two neighbouring 16-byte chunks of the row, which the swizzle keeps in one
    // 32-byte sector (odd rows in exchanged order): one store each
    const int64_t at = dst + (piece >> 2) * SLAB + row * 128 + (((2 * (piece & 3)) ^ (row & 6)) * 16);
    uint32_t ko[8], vo[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t u = vw[c] ^ 0x80808080u;
      ko[2 * c] = sizeof(T) == 4 ? pair_f16(kw[c] ^ 0x80808080u, 0x4140) : pair_bf16(kw[c], 0x4140);
      ko[2 * c + 1] = sizeof(T) == 4 ? pair_f16(kw[c] ^ 0x80808080u, 0x4342) : pair_bf16(kw[c], 0x4342);
      vo[2 * c] = pair_f16(u, 0x4140);
      vo[2 * c + 1] = pair_f16(u, 0x4342);
    }
    store32(p.kx + at, ko, row & 1);
    store32(p.vx + at, vo, row & 1);
  }
}

// ---- shared pieces --------------------------------------------------------------------------
// Row r of the tile whose first query is j0 (may be negative: the first tile is cut short).
struct Row {
  int j, g;
  bool on;
};
__device__ __forceinline__ Row row_of(const Kv8Tc& p, int j0, int r) {
  Row x;
  const int jl = r * p.g_magic >> 16;
  x.j = j0 + jl;
  x.g = r - jl * p.G;
  x.on = jl < p.qpt && x.j >= 0;
  return x;
}

// Gathers a tile's query rows into swizzled slabs with 16-byte asynchronous copies (rows that
// do not exist are zero); the caller waits for them and fences.
template <int HD>
__device__ __forceinline__ void gather_q(const Kv8Tc& p, int s, int h, int j0, uint8_t* dst, int tid, int n_thr) {
  constexpr int PER = HD / 8;              // 16-byte pieces in a row; n_thr is a multiple of it
  const int piece = tid % PER;
  const bf16* q = static_cast<const bf16*>(p.q) + ((int64_t)s * p.n_q * p.H + (int64_t)h * p.G) * HD + piece * 8;
  for (int r = tid / PER; r < BM; r += n_thr / PER) {
    const Row x = row_of(p, j0, r);
    const bf16* src = q + ((int64_t)(x.on ? x.j : 0) * p.H + (x.on ? x.g : 0)) * HD;
    const uint32_t d = tc::smem_u32(dst + (piece >> 3) * SLAB + r * 128 + (((piece & 7) ^ (r & 7)) * 16));
    const int bytes = x.on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
  }
}
// The same for fp32 queries, two threads per row: the row divided by a power of two (to rf; its
// largest magnitude is then in [1, 2)) as two fp16 parts, one tile after the other.  rf >= 2^-120
// keeps a score's factor rf ks log2(e) / sqrt(hd) above 0 (2^-149.55 at the least, hd 128 and ks
// 1e-8, which rounds up to 2^-149): an unseen score of -inf times 0 would be NaN.
template <int HD>
__device__ __forceinline__ void split_q(const Kv8Tc& p, int s, int h, int j0, uint8_t* dst, float* rf, int tid) {
  const int r = tid >> 1, half = tid & 1;
  const Row x = row_of(p, j0, r);
  const float* src = static_cast<const float*>(p.q) +
                     (((int64_t)s * p.n_q + (x.on ? x.j : 0)) * p.H + (int64_t)h * p.G + (x.on ? x.g : 0)) * HD + half * (HD / 2);
  float amax = 0.f;
#pragma unroll 4
  for (int c = 0; c < HD / 2; c += 4) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (x.on) ld4(src + c, f);
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  int e = amax > 0.f ? ilogbf(amax) : 0;
  e = e < -120 ? -120 : (e > 120 ? 120 : e);
  const float down = ldexpf(1.0f, -e);
  if (half == 0) rf[r] = ldexpf(1.0f, e);
#pragma unroll 2
  for (int c = 0; c < HD / 16; ++c) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (x.on) {
      ld4(src + c * 8, f);
      ld4(src + c * 8 + 4, f + 4);
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[2 * i] * down, b = f[2 * i + 1] * down;
      hi[i] = pack_h2(a, b);
      lo[i] = rest_h2(a, b, hi[i]);
    }
    const int chunk = half * (HD / 16) + c;
    uint8_t* d = dst + (chunk >> 3) * SLAB + r * 128 + (((chunk & 7) ^ (r & 7)) * 16);
    *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(d + HD / 64 * SLAB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---- attention ------------------------------------------------------------------------------
template <int HD, bool FUSED, typename T>
struct Layout {
  static constexpr int T_BYTES = HD / 64 * SLAB;             // a tile of Q, K or V
  static constexpr int Q_BYTES = parts<T>() * T_BYTES;
  static constexpr int C_BYTES = FUSED ? BN * HD : 0;        // a tile of codes
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = Q_BYTES;                      // [2 groups]
  static constexpr int OFF_V = OFF_K + 2 * T_BYTES;          // [2]
  static constexpr int OFF_C = OFF_V + 2 * T_BYTES;          // [2 groups][K, V] codes; the row statistics come there
                                                             // after the last ones are used up
  static constexpr int OFF_X = OFF_C;                        // [2 groups][2][BM] row max, row sum
  static constexpr int OFF_ML = OFF_X + 4 * BM * 4;          // [2][BM] the CTA's row max and sum, read by the cluster
  static constexpr int OFF_SC = FUSED ? OFF_C + 4 * C_BYTES : OFF_ML + 2 * BM * 4;   // [NSOFT][NG] float4 {ks, log2 vs, 1/vs, -}
  static constexpr int OFF_BAR = OFF_SC + NSOFT * NG * 16;
  static constexpr int SMEM = OFF_BAR + 128 + 1024 > tc::kWholeSm ? OFF_BAR + 128 + 1024 : tc::kWholeSm;
  static_assert(OFF_ML + 2 * BM * 4 <= OFF_SC, "the row statistics exceed the codes");
  static_assert(BM * HD * 4 <= 4 * T_BYTES, "the merge buffer exceeds K and V");
  static_assert(SMEM <= 227 * 1024, "shared memory exceeds the per-block limit");
};
constexpr uint32_t TM_O = 2 * BN;    // O_0 at column 256, O_1 right after it

// A warp's scales of one key tile: lane l < NG loads group l's pair (1 past the visible keys:
// the block may never have been written).
struct Scales {
  float k, v;
};
__device__ __forceinline__ Scales load_scales(const float* ks, const float* vs, int lg, int tile, int64_t nk, int lane) {
  Scales r{1.0f, 1.0f};
  const int64_t key = (int64_t)tile * BN + 16 * lane;
  if (lane < NG && key < nk) {
    r.k = ks[key >> lg];
    r.v = vs[key >> lg];
  }
  return r;
}

// A tile's codes as an operand tile, by a group's 128 threads: 16 codes at a time to two 16-byte
// words of the swizzled row.  Eight lanes take half a row of 64 channels each of two rows, so that
// their writes meet all banks; a thread's rows lie a multiple of 8 apart, so its addresses differ
// by constants.
template <int HD, bool IS_V>
__device__ __forceinline__ void convert_tile(const uint8_t* codes, uint8_t* dst, unsigned t) {
  constexpr int ROWS_AT_ONCE = 128 * 16 / HD;
  // lanes of a row pair: 4 of one row, 4 of the other, then (HD = 128) the same of the second slab
  const unsigned slab = HD == 128 ? (t >> 3) & 1 : 0, pair = HD == 128 ? t >> 4 : t >> 3;
  const unsigned row = 2 * pair + ((t >> 2) & 1), piece = t & 3, sw = row & 7;
  const uint8_t* src = codes + row * HD + slab * 64 + piece * 16;
  uint8_t* d0 = dst + slab * SLAB + row * 128 + ((2 * piece) ^ sw) * 16;
  uint8_t* d1 = dst + slab * SLAB + row * 128 + ((2 * piece + 1) ^ sw) * 16;
#pragma unroll 4
  for (int i = 0; i < BN / ROWS_AT_ONCE; ++i) {
    const uint4 u = *reinterpret_cast<const uint4*>(src + i * ROWS_AT_ONCE * HD);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint4 o;
      if (IS_V) {
        const uint32_t u0 = w[2 * c] ^ 0x80808080u, u1 = w[2 * c + 1] ^ 0x80808080u;
        o = make_uint4(pair_f16(u0, 0x4140), pair_f16(u0, 0x4342), pair_f16(u1, 0x4140), pair_f16(u1, 0x4342));
      } else {
        o = make_uint4(pair_bf16(w[2 * c], 0x4140), pair_bf16(w[2 * c], 0x4342), pair_bf16(w[2 * c + 1], 0x4140),
                       pair_bf16(w[2 * c + 1], 0x4342));
      }
      *reinterpret_cast<uint4*>((c ? d1 : d0) + i * ROWS_AT_ONCE * 128) = o;
    }
  }
}

// The largest t of a row's 128 scores.
template <typename T>
__device__ __forceinline__ float row_max(const uint32_t* sr, const float4* sc, float rf) {
  float mt = -INFINITY;
#pragma unroll
  for (int gg = 0; gg < NG; ++gg) {
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const uint32_t* x = sr + gg * 16 + i;
      a = fmax3(a, __uint_as_float(x[0]), __uint_as_float(x[1]));
      b = fmax3(b, __uint_as_float(x[2]), __uint_as_float(x[3]));
    }
    const float4 c = sc[gg];
    mt = fmaxf(mt, fmaf(fmaxf(a, b), sizeof(T) == 4 ? c.x * rf : c.x, c.y));
  }
  return mt;
}
// P = 2^(t - m + bias) over S as fp16 pairs (keys 2w, 2w + 1 to column w; fp32: the parts left over
// by the rounding 64 columns on), and its sum with 1 / vs; an unseen score of -inf gives 0.
template <typename T>
__device__ __forceinline__ float row_weights(const uint32_t* sr, uint32_t tS, const float4* sc, float off, float rf) {
  float l = 0.f;
#pragma unroll
  for (int c = 0; c < NG / 2; ++c) {
    uint32_t pk[16], lo[16];
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
      const float4 k = sc[2 * c + gg];
      const float f = sizeof(T) == 4 ? k.x * rf : k.x;
      const uint64_t f2 = f2_pack(f, f), a2 = f2_pack(k.y + off, k.y + off);
      uint64_t sum = 0ull;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const int k0 = c * 32 + gg * 16 + 2 * w;
        const float2 z = f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[k0]), __uint_as_float(sr[k0 + 1])), f2, a2));
        const float p0 = tc::ex2_approx(z.x), p1 = tc::ex2_approx(z.y);
        sum = f2_add(sum, f2_pack(p0, p1));
        pk[gg * 8 + w] = pack_h2(p0, p1);
        if constexpr (sizeof(T) == 4) lo[gg * 8 + w] = rest_h2(p0, p1, pk[gg * 8 + w]);
      }
      const float2 sm = f2_unpack(sum);
      l = fmaf(sm.x + sm.y, k.z, l);
    }
    tc::tmem_st16u_nowait(tS + c * 16, pk);
    if constexpr (sizeof(T) == 4) tc::tmem_st16u_nowait(tS + BN / 2 + c * 16, lo);
  }
  return l;
}

// Two groups of four warps take alternate key tiles (TMEM: S_0 | S_1 | O_0 | O_1), merged at
// the end; a cluster's CTAs take consecutive runs of key tiles.  A group is a closed loop: its
// first warp issues its copies and products between its share of the softmax, so a tile's chain
// is S -> softmax -> P V -> S of the next tile with one hand-over each way, the other group
// fills the gaps, and the eight warps (two per scheduler) may hold a row's 128 scores in
// registers and read them once.  K's buffer is refilled as soon as S is there, V's once P V is
// done: each load has most of a tile's chain to arrive, so one buffer per group suffices.
// Measured (3328 rows of 56 heads over 16384 rows of 8, 973 GFLOP): 801 us, 1.21 PFLOP/s, bound
// by the loop's hand-overs and products (without any softmax 698 us), at 1370 of 1400 W.  With a
// copying and an issuing warp, a ring of five tiles and the scores read twice for want of
// registers 1023 us; with one accumulator, S two tiles ahead and the maximum handed on from tile to
// tile 883 us; with half tiles and two score buffers per group 949 us; with two query tiles per CTA
// on shared key tiles 879 us.
//
// FUSED: the operands do not come ready from k_kv8_expand; the group that uses a tile converts it
// itself, K while P V of the tile before runs, V while S runs.  That lengthens the loop by a half,
// but where only one query tile reads the keys it saves writing and reading four bytes per code:
// 85 rows of 40 heads over 6 x 16064 keys (987 MB of codes) 388 us instead of 651, 118 of 32 heads
// over 1664 keys 16.5 instead of 21; with three query tiles (299 rows, 32 heads, 13440 keys) 182
// instead of 163.
template <int HD, bool FUSED, typename T>
__global__ void __launch_bounds__(ATTN_THREADS, 1) k_kv8_attn_tc(const Kv8Tc p, int n_split) {
  pdl_wait();
  pdl_trigger();                   // (before TMEM is allocated: see tc::kWholeSm; after it 62.2 us instead of 61.8 at 7B)
  using L = Layout<HD, FUSED, T>;
  constexpr int NP = parts<T>(), RW = row_words<T>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = base + L::OFF_Q;
  float* xm = reinterpret_cast<float*>(base + L::OFF_X);   // [2][BM] row max, then [2][BM] row sum
  float* xl = xm + 2 * BM;
  float* cm = reinterpret_cast<float*>(base + L::OFF_ML);  // [BM] max, [BM] sum
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
  uint64_t* k_full = bars + 5 * grp;       // a group's barriers: K and V have landed, S and P V are done,
  uint64_t* v_full = k_full + 1;
  uint64_t* s_full = k_full + 2;
  uint64_t* pv_done = k_full + 3;
  uint64_t* v_empty = k_full + 4;          // the four warps have read V's codes
  const int rank = blockIdx.x % n_split, h = blockIdx.x / n_split, s = blockIdx.z;
  // tiles are cut from the end of the queries: the longest rows come first, and the tile that
  // is cut short is the one with the lowest positions
  const int j0 = p.n_q - (int)(blockIdx.y + 1) * p.qpt;
  const int64_t head = (int64_t)s * p.Hkv + h;

  if (tid == 0) {
    for (int i = 0; i < 10; ++i) tc::mbar_init(&bars[i], i % 5 == 4 ? 4 : 1);
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, TMEM_COLS);
    tc::tmem_relinquish();
  }
  if constexpr (NP == 2)
    split_q<HD>(p, s, h, j0, sQ, cm, tid);
  else
    gather_q<HD>(p, s, h, j0, sQ, tid, ATTN_THREADS);
  // keys that some row of the tile sees
  int mx = -1;
  for (int i = tid; i < p.qpt; i += ATTN_THREADS) {
    const int j = j0 + i;
    if (j >= 0) {
      const int l = p.last[(int64_t)s * p.n_q + j];
      if ((l < -1 || l >= p.c.capacity) && rank == 0) atomicOr(&g_err_kv8_tc, ERRBIT_INDEX);
      mx = max(mx, last_of(p, s, j));
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  int* wm = reinterpret_cast<int*>(xm);
  if (lane == 0) wm[warp] = mx;
  cp_async_wait_all();
  tc::fence_proxy_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
#pragma unroll
  for (int w = 0; w < ATTN_THREADS / 32; ++w) mx = max(mx, wm[w]);
  const float rf = NP == 2 ? cm[r] : 1.0f;
  __syncthreads();                 // wm's memory is the groups' row maxima later on, cm's the CTA's
  // For the weights a query that sees nothing is a row of zeros like one that does not exist: it may
  // hold a NaN or an infinity, whose scores the weights' mask-free sum could not tell from others.
  // (Comparing every key with -1 there instead: 85 padded rows x 6, 40 heads, 661 us instead of 650.)
  if (p.weights) {
    const Row y = row_of(p, j0, tid >> 1);
    if (y.on && last_of(p, s, y.j) < 0)
#pragma unroll 1
      for (int i = tid & 1; i < L::Q_BYTES / SLAB * 8; i += 2)
        *reinterpret_cast<uint4*>(sQ + (i >> 3) * SLAB + (tid >> 1) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    __syncthreads();
  }
  // for the weights: the tile's queries as they sit in shared memory, and its bound
  const int64_t qt = head * p.q_tiles + blockIdx.y;
  if (p.weights && rank == 0 && tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p.qx + qt * L::Q_BYTES),
                 "r"(tc::smem_u32(sQ)), "r"((uint32_t)L::Q_BYTES)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    if (h == 0) p.tile_max[(int64_t)s * p.q_tiles + blockIdx.y] = mx;
  }
  const int64_t nk = (int64_t)mx + 1;
  const int all = (mx + BN) / BN;  // key tiles; 0 if no row sees a key
  const int ta = (int)((int64_t)all * rank / n_split), n_kt = (int)((int64_t)all * (rank + 1) / n_split) - ta;
  const int nt = n_kt > grp ? (n_kt - grp + 1) / 2 : 0;     // this group's: ta + grp, ta + grp + 2, ...

  const Row x = row_of(p, j0, r);
  const int last = x.on ? last_of(p, s, x.j) : -1;
  const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const uint32_t tS = trow + grp * BN, tO = trow + TM_O + grp * HD;
  bool ok = true;                  // of this warp; one that gave up goes on meeting its group
  {
    const bool issuer = quad == 0;
    uint8_t* sK = base + L::OFF_K + grp * L::T_BYTES;
    uint8_t* sV = base + L::OFF_V + grp * L::T_BYTES;
    uint8_t* cK = base + L::OFF_C + grp * 2 * L::C_BYTES;
    uint8_t* cV = cK + L::C_BYTES;
    int nk_loads = 0, nv_loads = 0;
    auto load = [&](const uint8_t* tiles, const int8_t* codes, uint8_t* dst, uint8_t* cdst, uint64_t* bar, int u) {
      if (lane != 0) return;
      const int tile = ta + grp + 2 * u;
      if constexpr (FUSED) {
        const int64_t key = (int64_t)tile * BN;
        const uint32_t bytes = (uint32_t)(p.c.capacity - key < BN ? p.c.capacity - key : BN) * HD;
        tc::mbar_expect_tx(bar, bytes);
        tc::bulk_load(cdst, codes + (head * p.c.capacity + key) * HD, bytes, bar);
      } else {
        tc::mbar_expect_tx(bar, L::T_BYTES);
        tc::bulk_load(dst, tiles + (head * p.tiles + tile) * (int64_t)L::T_BYTES, L::T_BYTES, bar);
      }
    };
    auto load_k = [&](int u) {
      ++nk_loads;
      load(p.kx, p.c.k_codes, sK, cK, k_full, u);
    };
    auto load_v = [&](int u) {
      ++nv_loads;
      load(p.vx, p.c.v_codes, sV, cV, v_full, u);
    };
    auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory"); };
    auto issue_s = [&]() {
      constexpr uint32_t idesc = NP == 2 ? tc::idesc_f16_f32(BM, BN) : tc::idesc_bf16_f32(BM, BN);
      const uint64_t qd = tc::desc_sw128(tc::smem_u32(sQ)), kd = tc::desc_sw128(tc::smem_u32(sK));
      tc::tc_fence_after();
      if (tc::elect_one()) {
#pragma unroll
        for (int part = 0; part < NP; ++part)
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t off = ((k >> 2) * SLAB + (k & 3) * 32) >> 4;
            tc::mma_bf16(tmem + grp * BN, qd + ((part * L::T_BYTES) >> 4) + off, kd + off, idesc, part + k > 0);
          }
        tc::mma_commit(s_full);
      }
      __syncwarp();
    };
    auto issue_pv = [&](bool add) {
      constexpr uint32_t idesc = tc::idesc_f16_f32(BM, HD, true);
      const uint64_t vd = tc::desc_sw128_mn(tc::smem_u32(sV), SLAB);
      tc::tc_fence_after();
      if (tc::elect_one()) {
#pragma unroll
        for (int part = 0; part < NP; ++part)
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            tc::mma_bf16_ts(tmem + TM_O + grp * HD, tmem + grp * BN + part * (BN / 2) + k * 8,
                            vd + (uint64_t)((k * 16 * 128) >> 4), idesc, (add || part + k > 0) ? 1u : 0u);
        tc::mma_commit(pv_done);
      }
      __syncwarp();
    };
    const int64_t nblk = p.c.capacity >> p.lg;
    const float* ks = p.c.k_scale + head * nblk;
    const float* vs = p.c.v_scale + head * nblk;
    float4* sc = reinterpret_cast<float4*>(base + L::OFF_SC) + warp * NG;
    float m_used = -INFINITY, l = 0.f;
    Scales nx = load_scales(ks, vs, p.lg, ta + grp, nk, lane);
    // softmax of the group's tile u: scores to P, in place; on_scores() runs once they are there
    auto softmax = [&](int u, auto&& on_scores) {
      const int tile = ta + grp + 2 * u;
      __syncwarp();
      if (lane < NG) {
        const float v = fmaxf(nx.v, kKv8MinScale);
        // (approximate log and reciprocal: off by 2 ulp, which for the log is 2^-20 at vs = 0.03 and
        // 2^-18 at the smallest scale, absolute in P's exponent, beside P's own rounding of 2^-12; the
        // exact forms cost 40 of 850 us at the Yi shape, by the few lanes that compute them)
        sc[lane] = make_float4(fmaxf(nx.k, kKv8MinScale) * p.scale_log2, NP == 2 ? log2f(v) : __log2f(v), __fdividef(1.0f, v), 0.f);
      }
      nx = load_scales(ks, vs, p.lg, tile + 2, nk, lane);
      __syncwarp();
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(s_full, u & 1));
      if (!ok) return;
      on_scores();
      uint32_t sr[BN];
      tc::tc_fence_after();
#pragma unroll
      for (int c = 0; c < BN; c += 32) tc::tmem_ld32_nowait(tS + c, sr + c);
      tc::tmem_wait_ld64(sr);
      tc::tmem_wait_ld64(sr + 64);
      const int seen = last - tile * BN;     // the last key of the tile that the row sees
      if (__any_sync(0xffffffffu, seen < BN - 1)) {          // most tiles are seen whole by all rows of the warp
#pragma unroll
        for (int i = 0; i < BN; ++i)
          if (i > seen) sr[i] = 0xff800000u;
      }
      const float mt = row_max<T>(sr, sc, rf);
      if (u == 0) {
        m_used = mt;             // O_g is written, not added to, by this tile's P V
      } else {
        const bool need = mt > m_used + kLazy;
        if (__any_sync(0xffffffffu, need)) {                 // (S was issued after the last P V had completed)
          const float alpha = need ? tc::ex2_approx(m_used - mt) : 1.0f;
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            float o[16];
            tc::tmem_ld16(tO + c * 16, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tc::tmem_st16(tO + c * 16, o);
          }
          l *= alpha;
          if (need) m_used = mt;
        }
      }
      l += row_weights<T>(sr, tS, sc, kPBias - (m_used == -INFINITY ? 0.f : m_used), rf);
      tc::tmem_wait_st();
      tc::tc_fence_before();
    };
    if (issuer && nt > 0) {
      load_k(0);
      load_v(0);
    }
    if constexpr (FUSED) {
#pragma unroll 1
      for (int u = -1; u < nt; ++u) {
        if (u >= 0) {
          softmax(u, [] {});
          group_sync();            // P is there, and V, converted while S was on its way
          if (issuer && ok) issue_pv(u > 0);
        }
        if (u + 1 >= nt) break;
        // K of the next tile while P V runs: S of this tile is done with its buffer
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(k_full, (u + 1) & 1));
        if (ok) convert_tile<HD, false>(cK, sK, r);
        tc::fence_proxy_async_smem();
        group_sync();
        // S goes where P is, and V's buffer is free, once P V is done
        ok = ok && (u < 0 || __all_sync(0xffffffffu, tc::mbar_wait(pv_done, u & 1)));
        if (issuer && ok) {
          issue_s();
          if (u + 2 < nt) load_k(u + 2);
        }
        // V of the next tile while S runs
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(v_full, (u + 1) & 1));
        if (ok) convert_tile<HD, true>(cV, sV, r);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(v_empty);
        if (issuer && u + 2 < nt) {
          ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(v_empty, (u + 1) & 1));
          if (ok) load_v(u + 2);
        }
      }
    } else {
      if (issuer && nt > 0) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(k_full, 0));
        if (ok) issue_s();
      }
#pragma unroll 1
      for (int u = 0; u < nt; ++u) {
        softmax(u, [&] {
          if (issuer && u + 1 < nt) load_k(u + 1);
        });
        group_sync();
        if (issuer) {
          ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(v_full, u & 1));
          if (ok) issue_pv(u > 0);
          if (u + 1 < nt) {
            ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(k_full, (u + 1) & 1) && tc::mbar_wait(pv_done, u & 1));
            if (ok) {
              issue_s();
              load_v(u + 1);
            }
          }
        }
      }
    }
    ok = ok && (nt == 0 || __all_sync(0xffffffffu, tc::mbar_wait(pv_done, (nt - 1) & 1)));
    if (!ok) {
      // report, and give the copies in flight as long again before the memory is given up
      if (lane == 0) atomicOr(&g_err_kv8_tc, ERRBIT_TIMEOUT);
      if (nk_loads > 0) tc::mbar_wait(k_full, (nk_loads - 1) & 1);
      if (nv_loads > 0) tc::mbar_wait(v_full, (nv_loads - 1) & 1);
    }
    if (FUSED) __syncthreads();    // the statistics go where the other group's codes may still be
    // both groups' row statistics meet in shared memory
    xm[grp * BM + r] = m_used;
    xl[grp * BM + r] = l;
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const float ma = xm[r], mb = xm[BM + r], mm = fmaxf(ma, mb);
    const float a0 = ma == -INFINITY ? 0.f : tc::ex2_approx(ma - mm);
    const float a1 = mb == -INFINITY ? 0.f : tc::ex2_approx(mb - mm);
    const float lt = xl[r] * a0 + xl[BM + r] * a1;
    const float inv = lt > 0.f ? 1.0f / lt : 0.f;
    if (grp == 0) {
      if (n_split > 1) {
        cm[r] = isnan(lt) ? lt : mm;       // (a NaN's scores leave no maximum; the row is not to look empty)
        cm[BM + r] = lt;
      } else if (p.weights) {
        p.rows[qt * RW * BM + r] = lt == 0.f ? INFINITY : mm - kPBias + log2f(lt);
      }
      if (p.weights && rank == 0) {
        p.rows[qt * RW * BM + BM + r] = __int_as_float(last);
        if (NP == 2) p.rows[qt * RW * BM + 2 * BM + r] = rf;
      }
    }
    // group g finalises columns [g HD/2, (g + 1) HD/2); O_g was never written with fewer than
    // g + 1 key tiles
    float* om = reinterpret_cast<float*>(base + L::OFF_K) + r * HD;
    T* orow = static_cast<T*>(p.out) + (((int64_t)s * p.n_q + (x.on ? x.j : 0)) * p.H + (int64_t)h * p.G + (x.on ? x.g : 0)) * HD;
#pragma unroll 1
    for (int c = 0; c < HD / 32; ++c) {
      const int col = grp * (HD / 2) + c * 16;
      float o0[16], o1[16];
      if (n_kt > 0) {
        tc::tmem_ld16(trow + TM_O + col, o0);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) o0[i] = 0.f;
      }
      if (n_kt > 1) {
        tc::tmem_ld16(trow + TM_O + HD + col, o1);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) o1[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o0[i] = o0[i] * a0 + o1[i] * a1;
      if (n_split > 1) {
        // 16-byte words rotated by the row, so that the rows of a warp spread over the banks
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(om + (((col >> 2) + i) ^ (r & 7)) * 4) =
              make_float4(o0[4 * i], o0[4 * i + 1], o0[4 * i + 2], o0[4 * i + 3]);
      } else if (x.on) {
#pragma unroll
        for (int i = 0; i < 16; ++i) o0[i] *= inv;
        st8(orow + col, o0);
        st8(orow + col + 8, o0 + 8);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (n_split > 1) {
    // ------------------------------------------------------------------ merge of the cluster
    tc::cluster_sync();
    const uint32_t cm_a = tc::smem_u32(cm), om_a = tc::smem_u32(base + L::OFF_K);
    const int per = (BM + n_split - 1) / n_split, r0 = rank * per, nr = min(per, BM - r0);   // this CTA's share of the rows
    constexpr int W4 = HD / 4;
    for (int i = tid; i < nr * W4; i += ATTN_THREADS) {
      const int r = r0 + i / W4, w = i % W4;
      const Row x = row_of(p, j0, r);
      float M = -INFINITY, sum = 0.f;
      for (int c = 0; c < n_split; ++c) M = fmaxf(M, tc::ld_cluster(tc::mapa_shared(cm_a + 4 * r, c)));
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < n_split; ++c) {
        const float mc = tc::ld_cluster(tc::mapa_shared(cm_a + 4 * r, c));
        if (mc == -INFINITY) continue;
        const float f = tc::ex2_approx(mc - M);
        sum = fmaf(tc::ld_cluster(tc::mapa_shared(cm_a + 4 * (BM + r), c)), f, sum);
        const float4 v = tc::ld_cluster4(tc::mapa_shared(om_a + 4 * (r * HD + (w ^ (r & 7)) * 4), c));
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
        o[2] = fmaf(v.z, f, o[2]);
        o[3] = fmaf(v.w, f, o[3]);
      }
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] *= inv;
      if (x.on) st4(static_cast<T*>(p.out) + (((int64_t)s * p.n_q + x.j) * p.H + (int64_t)h * p.G + x.g) * HD + 4 * w, o);
      // (as without a split: +inf only for a row that sees nothing, a NaN row's is NaN)
      if (p.weights && w == 0) p.rows[qt * RW * BM + r] = sum == 0.f ? INFINITY : M - kPBias + log2f(sum);
    }
    tc::cluster_sync();            // the peers may still be reading this CTA's part
  }
  if (p.weights && rank == 0 && tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (warp == 0) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---- weights --------------------------------------------------------------------------------
// S^T = C_K Q^T puts a key in each TMEM lane, so the sum over the query rows stays inside a
// thread.  A resident CTA takes pairs of key tiles (of one KV head and sequence), one per
// softmax group, and streams the query tiles that see them past both: a query tile is loaded
// once for 256 keys, each group has two S buffers (TMEM 4 x 128 columns), and no sums have to
// meet.  Warp roles: 0 = copies, 1 = TMEM allocation and MMA issue, 2..9 = softmax.
// Measured: 64 queries of 7 heads over 16384 rows of 8 KV heads (58.7 M weights) 21 us, bound by
// the exponentials' chain from TMEM (33% of the issue slots, 32% of the special functions' rate);
// one CTA per key tile gathering the queries itself 55 us.
//
// FUSED (one query tile): K comes as codes, and a group converts the next pair's tile as soon as S of
// this one's has come, before it weighs (85 rows of 40 heads over 6 x 16064 keys, attention and
// weights 650 us; converting after weighing 681, with the expansion 842).
template <int HD, bool FUSED, typename T>
struct WLayout {
  static constexpr int T_BYTES = HD / 64 * SLAB;
  static constexpr int C_BYTES = FUSED ? BN * HD : 0;
  static constexpr int Q_BYTES = parts<T>() * T_BYTES;
  static constexpr int L_BYTES = row_words<T>() * BM * 4;
  static constexpr int QS = FUSED || parts<T>() == 2 ? 2 : 4; // query tiles in flight
  static constexpr int OFF_K = 0;                             // [2]
  static constexpr int OFF_Q = 2 * T_BYTES;                   // [QS]
  static constexpr int OFF_C = OFF_Q + QS * Q_BYTES;          // [2] codes
  static constexpr int OFF_L = OFF_C + 2 * C_BYTES;           // [QS][row_words][BM] log2 sum, last, power of two
  static constexpr int OFF_BAR = OFF_L + QS * L_BYTES;
  static constexpr int SMEM = OFF_BAR + 256 + 1024 > tc::kWholeSm ? OFF_BAR + 256 + 1024 : tc::kWholeSm;
  static_assert(SMEM <= 227 * 1024, "shared memory exceeds the per-block limit");
};

// The query tiles that see a pair of key tiles, in ascending order, 32 bounds at a time; every
// role of the CTA walks the same list.
struct TileWalk {
  const int32_t* bound;     // of the sequence's query tiles
  int n, key0, base, lane;
  unsigned mask;
  __device__ __forceinline__ TileWalk(const int32_t* b, int n_, int key0_, int lane_)
      : bound(b), n(n_), key0(key0_), base(-32), lane(lane_), mask(0) {}
  // the next tile, -1 at the end
  __device__ __forceinline__ int next() {
    while (!mask) {
      base += 32;
      if (base >= n) return -1;
      mask = __ballot_sync(0xffffffffu, base + lane < n && bound[base + lane] >= key0);
    }
    const int y = base + __ffs(mask) - 1;
    mask &= mask - 1;
    return y;
  }
};

template <int HD, bool FUSED, typename T>
__global__ void __launch_bounds__(THREADS, 1) k_kv8_weights_tc(const Kv8Tc p) {
  using L = WLayout<HD, FUSED, T>;
  constexpr int NP = parts<T>(), RW = row_words<T>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sK = base + L::OFF_K;
  uint8_t* sQ = base + L::OFF_Q;
  const float* sL = reinterpret_cast<const float*>(base + L::OFF_L);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(base + L::OFF_BAR);   // [2] K (its codes) has landed
  uint64_t* k_empty = k_full + 2;                                       // [2] the products (the four warps) have read it
  uint64_t* k_conv = k_empty + 2;                                       // [2] the four warps have converted it
  uint64_t* q_full = k_conv + 2;                                        // [QS]
  uint64_t* q_empty = q_full + L::QS;                                   // [QS] the MMA and every softmax warp
  uint64_t* s_full = q_empty + L::QS;                                   // [2 groups][2]
  uint64_t* s_empty = s_full + 4;                                       // [2][2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_empty + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&k_full[i], 1);
      tc::mbar_init(&k_empty[i], FUSED ? 4 : 1);
      tc::mbar_init(&k_conv[i], 4);
    }
    for (int i = 0; i < L::QS; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1 + NSOFT);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&s_empty[i], 4);
    }
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int pairs = (p.tiles + 1) / 2;
  const int64_t items = (int64_t)p.c.n_seq * p.Hkv * pairs;
  struct Pair {
    int64_t it, head;
    int s, kt;            // sequence, first key tile
    bool two;             // a query sees the second
  };
  // this CTA's first pair from `it` on that a query sees
  auto find = [&](int64_t it, Pair& x) -> bool {
    for (; it < items; it += gridDim.x) {
      x.it = it;
      x.head = it / pairs;
      x.s = (int)(x.head / p.Hkv);
      x.kt = 2 * (int)(it - x.head * pairs);
      const int mx = p.seq_max[x.s];
      if (x.kt * BN > mx) continue;
      x.two = x.kt + 1 < p.tiles && (x.kt + 1) * BN <= mx;
      return true;
    }
    return false;
  };
  auto each = [&](auto&& f) {
    Pair x;
    for (bool more = find(blockIdx.x, x); more; more = find(x.it + gridDim.x, x))
      if (!f(x.head, x.s, x.kt, x.two)) break;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ copies
    bool ok = true;
    int n = 0, kn[2] = {0, 0};
    each([&](int64_t head, int s, int kt, bool two) -> bool {
      for (int g = 0; ok && g < (two ? 2 : 1); ++g) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&k_empty[g], (kn[g] & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          if constexpr (FUSED) {
            const int64_t key = (int64_t)(kt + g) * BN;
            const uint32_t bytes = (uint32_t)(p.c.capacity - key < BN ? p.c.capacity - key : BN) * HD;
            tc::mbar_expect_tx(&k_full[g], bytes);
            tc::bulk_load(base + L::OFF_C + g * L::C_BYTES, p.c.k_codes + (head * p.c.capacity + key) * HD, bytes, &k_full[g]);
          } else {
            tc::mbar_expect_tx(&k_full[g], L::T_BYTES);
            tc::bulk_load(sK + g * L::T_BYTES, p.kx + (head * p.tiles + kt + g) * (int64_t)L::T_BYTES, L::T_BYTES, &k_full[g]);
          }
        }
        ++kn[g];
      }
      TileWalk walk(p.tile_max + (int64_t)s * p.q_tiles, p.q_tiles, kt * BN, lane);
      for (int y; ok && (y = walk.next()) >= 0; ++n) {
        const int b = n % L::QS;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_empty[b], ((n / L::QS) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          const int64_t qt = head * p.q_tiles + y;
          tc::mbar_expect_tx(&q_full[b], L::Q_BYTES + L::L_BYTES);
          tc::bulk_load(sQ + b * L::Q_BYTES, p.qx + qt * L::Q_BYTES, L::Q_BYTES, &q_full[b]);
          tc::bulk_load(base + L::OFF_L + b * L::L_BYTES, p.rows + qt * RW * BM, L::L_BYTES, &q_full[b]);
        }
        __syncwarp();
      }
      return ok;
    });
    if (!ok && lane == 0) atomicOr(&g_err_kv8_tc, ERRBIT_TIMEOUT);
    // no copy is in flight when the CTA ends, whoever gave up on what
    for (int g = 0; g < 2; ++g)
      if (kn[g] > 0) tc::mbar_wait(&k_full[g], (kn[g] - 1) & 1);
    for (int i = n > L::QS ? n - L::QS : 0; i < n; ++i) tc::mbar_wait(&q_full[i % L::QS], (i / L::QS) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue
    constexpr uint32_t idesc = NP == 2 ? tc::idesc_f16_f32(BN, BM) : tc::idesc_bf16_f32(BN, BM);
    const uint64_t k_desc = tc::desc_sw128(tc::smem_u32(sK)), q_desc = tc::desc_sw128(tc::smem_u32(sQ));
    bool ok = true;
    int n = 0, kn[2] = {0, 0}, sn[2] = {0, 0};
    each([&](int64_t, int s, int kt, bool two) -> bool {
      const int ng = two ? 2 : 1;
      for (int g = 0; ok && g < ng; ++g) ok = __all_sync(0xffffffffu, tc::mbar_wait(FUSED ? &k_conv[g] : &k_full[g], kn[g]++ & 1));
      TileWalk walk(p.tile_max + (int64_t)s * p.q_tiles, p.q_tiles, kt * BN, lane);
      for (int y = walk.next(); ok && y >= 0; ++n) {
        const int b = n % L::QS, ahead = walk.next();
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_full[b], (n / L::QS) & 1));
        for (int g = 0; ok && g < ng; ++g) {
          const int sb = sn[g] & 1;
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_empty[2 * g + sb], ((sn[g] >> 1) & 1) ^ 1));
          if (!ok) break;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint64_t kd = k_desc + (uint64_t)((g * L::T_BYTES) >> 4), qd = q_desc + (uint64_t)((b * L::Q_BYTES) >> 4);
#pragma unroll
            for (int part = 0; part < NP; ++part)
#pragma unroll
              for (int k = 0; k < HD / 16; ++k) {
                const uint32_t off = ((k >> 2) * SLAB + (k & 3) * 32) >> 4;
                tc::mma_bf16(tmem + (2 * g + sb) * BM, kd + off, qd + ((part * L::T_BYTES) >> 4) + off, idesc, part + k > 0);
              }
            tc::mma_commit(&s_full[2 * g + sb]);
            if (g == ng - 1) tc::mma_commit(&q_empty[b]);
            if (!FUSED && ahead < 0) tc::mma_commit(&k_empty[g]);
          }
          __syncwarp();
          ++sn[g];
        }
        y = ahead;
      }
      return ok;
    });
    if (!ok && lane == 0) atomicOr(&g_err_kv8_tc, ERRBIT_TIMEOUT);
  } else {
    // ------------------------------------------------------------------ softmax
    const int grp = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16) + grp * 2 * BM;
    bool ok = true;
    int n = 0, sn = 0, kn = 0;
    // K of a pair from its codes; the products of the pair before are done with it
    auto convert = [&](const Pair& x) {
      if (grp == 1 && !x.two) return;
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(&k_full[grp], kn & 1));
      if (!ok) return;
      ++kn;
      convert_tile<HD, false>(base + L::OFF_C + grp * L::C_BYTES, sK + grp * L::T_BYTES, r);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&k_empty[grp]);
        tc::mbar_arrive(&k_conv[grp]);
      }
    };
    // on_scores() runs each time S of this group's tile has come
    auto weigh = [&](int64_t head, int s, int kt, bool two, auto&& on_scores) -> bool {
      const bool mine = grp == 0 || two;
      const int key = (kt + grp) * BN + r;
      float f = 0.f;
      if (mine && key < p.c.capacity)
        f = fmaxf(p.c.k_scale[head * (p.c.capacity >> p.lg) + (key >> p.lg)], kKv8MinScale) * p.scale_log2;
      const uint64_t f2 = f2_pack(f, f);
      float sum = 0.f;
      TileWalk walk(p.tile_max + (int64_t)s * p.q_tiles, p.q_tiles, kt * BN, lane);
      while (ok && walk.next() >= 0) {
        const int b = n % L::QS;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&q_full[b], (n / L::QS) & 1));
        if (!ok) break;
        if (mine) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&s_full[2 * grp + (sn & 1)], (sn >> 1) & 1));
          if (!ok) break;
          on_scores();
          if (!ok) break;
          tc::tc_fence_after();
          const float* lse = sL + b * RW * BM;
          const int* last = reinterpret_cast<const int*>(lse + BM);
          // the tile's queries either all see this warp's last key, or each is compared, whatever its
          // sum (a NaN's score stays one beside +inf).  Rows that see nothing are zeros: they weigh 0.
          int lo = 0x7fffffff;
#pragma unroll
          for (int i = 0; i < BM / 32; ++i) {
            const int v = last[i * 32 + lane];
            lo = min(lo, v < 0 ? 0x7fffffff : v);
          }
          const bool full = __reduce_min_sync(0xffffffffu, lo) >= (kt + grp) * BN + quad * 32 + 31;
          const uint32_t tS = trow + (sn & 1) * BM;
#pragma unroll 1
          for (int c = 0; c < BM / 64; ++c) {
            uint32_t sr[64];
            tc::tmem_ld32_nowait(tS + c * 64, sr);
            tc::tmem_ld32_nowait(tS + c * 64 + 32, sr + 32);
            tc::tmem_wait_ld64(sr);
            uint64_t acc[2] = {0ull, 0ull};
            // scores of rows i, i + 1 (fp32: in the row's own power of two)
            auto scores = [&](int i) -> uint64_t {
              const uint64_t x = f2_pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
              if constexpr (NP == 2) {
                const float2 e = *reinterpret_cast<const float2*>(lse + 2 * BM + c * 64 + i);
                return f2_fma(x, f2_pack(e.x, e.y), 0ull);
              }
              return x;
            };
            if (full) {
#pragma unroll
              for (int i = 0; i < 64; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(lse + c * 64 + i);
                const float2 z0 = f2_unpack(f2_fma(scores(i), f2, f2_pack(-v.x, -v.y)));
                const float2 z1 = f2_unpack(f2_fma(scores(i + 2), f2, f2_pack(-v.z, -v.w)));
                acc[0] = f2_add(acc[0], f2_pack(tc::ex2_approx(z0.x), tc::ex2_approx(z0.y)));
                acc[1] = f2_add(acc[1], f2_pack(tc::ex2_approx(z1.x), tc::ex2_approx(z1.y)));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 64; i += 2) {
                const float2 v = *reinterpret_cast<const float2*>(lse + c * 64 + i);
                const int2 t = *reinterpret_cast<const int2*>(last + c * 64 + i);
                const float2 z = f2_unpack(f2_fma(scores(i), f2, f2_pack(-v.x, -v.y)));
                const float e0 = key <= t.x ? tc::ex2_approx(z.x) : 0.f, e1 = key <= t.y ? tc::ex2_approx(z.y) : 0.f;
                acc[(i >> 1) & 1] = f2_add(acc[(i >> 1) & 1], f2_pack(e0, e1));
              }
            }
            const float2 x = f2_unpack(f2_add(acc[0], acc[1]));
            sum += x.x + x.y;
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s_empty[2 * grp + (sn & 1)]);
          ++sn;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&q_empty[b]);
        ++n;
      }
      if (ok && mine && key < p.c.capacity && sum != 0.f) p.weights[head * p.c.capacity + key] += sum;
      return ok;
    };
    if constexpr (FUSED) {
      // one query tile, so S comes once per pair: then K is free for the next pair's, whose S
      // runs while this pair is weighed
      Pair x, nx;
      bool more = find(blockIdx.x, x);
      if (more) convert(x);
      while (ok && more) {
        const bool next = find(x.it + gridDim.x, nx);
        auto ahead = [&] {
          if (next) convert(nx);
        };
        if (grp == 1 && !x.two) ahead();
        if (!weigh(x.head, x.s, x.kt, x.two, ahead)) break;
        more = next;
        if (more) x = nx;
      }
    } else {
      each([&](int64_t head, int s, int kt, bool two) { return weigh(head, s, kt, two, [] {}); });
    }
    if (!ok && lane == 0) atomicOr(&g_err_kv8_tc, ERRBIT_TIMEOUT);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Per device and kernel, set once its shared-memory limit is: how many clusters of 1..8 of its CTAs
// run at once, and the SM count.  Guarded for calls from several threads.
struct TcDevice {
  int clusters[9];
  int sms;
};
std::mutex g_tc_mu;
TcDevice g_tc[64][6];        // (HD, T, FUSED)

template <typename F>
cudaError_t allow_smem(F* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
template <int HD, bool FUSED, typename T>
cudaError_t prepare_tc(int dev, TcDevice* out) {
  constexpr int which = (HD == 128 ? 0 : 3) + (sizeof(T) == 4 ? 2 : FUSED ? 1 : 0);
  std::lock_guard<std::mutex> g(g_tc_mu);
  const bool cached = dev >= 0 && dev < 64;
  if (cached && g_tc[dev][which].sms) {
    *out = g_tc[dev][which];
    return cudaSuccess;
  }
  cudaError_t e = allow_smem(k_kv8_attn_tc<HD, FUSED, T>, Layout<HD, FUSED, T>::SMEM);
  if (e == cudaSuccess) e = allow_smem(k_kv8_weights_tc<HD, FUSED, T>, WLayout<HD, FUSED, T>::SMEM);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, dev);
  for (int ns = 1; e == cudaSuccess && ns <= 8; ++ns) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ns);
    cfg.blockDim = dim3(ATTN_THREADS);
    cfg.dynamicSmemBytes = Layout<HD, FUSED, T>::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ns;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&out->clusters[ns], k_kv8_attn_tc<HD, FUSED, T>, &cfg);
  }
  if (e == cudaSuccess && cached) g_tc[dev][which] = *out;
  return e;
}

template <int HD, bool FUSED, typename T>
cudaError_t launch_variant(const Kv8Tc& p, cudaStream_t s) {
  int dev = 0;
  TcDevice d{};
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (e = prepare_tc<HD, FUSED, T>(dev, &d)) != cudaSuccess) return e;
  if (!FUSED &&
      (e = launch_k(k_kv8_expand<HD, T>, dim3(p.tiles, p.Hkv, p.c.n_seq), dim3(256), 0, s, p)) != cudaSuccess)
    return e;
  // the keys are split as far as all parts still run at once, and have two tiles each (64 queries of 8
  // x 7 heads over 16384 keys, 32 units, in 1 / 2 / 4 / 8 parts: 170, 102, 62, 94 us; 85 queries of 40
  // heads over 16064, 40 units, in 2 / 3: 124, 88 us; 48 of 8 x 4 over 4096, 16 units, in 4 / 8: 30, 24)
  const int64_t units = (int64_t)p.q_tiles * p.Hkv * p.c.n_seq;
  int ns = 8;
  while (ns > 1 && (units > d.clusters[ns] || 2 * ns > p.tiles)) --ns;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.Hkv * ns, p.q_tiles, p.c.n_seq);
  cfg.blockDim = dim3(ATTN_THREADS);
  cfg.dynamicSmemBytes = Layout<HD, FUSED, T>::SMEM;
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
  if ((e = cudaLaunchKernelEx(&cfg, k_kv8_attn_tc<HD, FUSED, T>, p, ns)) != cudaSuccess || !p.weights) return e;
  const int64_t items = (int64_t)p.c.n_seq * p.Hkv * ((p.tiles + 1) / 2);
  return launch_k(k_kv8_weights_tc<HD, FUSED, T>, dim3((unsigned)(items < d.sms ? items : d.sms)), dim3(THREADS),
                  WLayout<HD, FUSED, T>::SMEM, s, p);
}

template <int HD, typename T>
cudaError_t launch_hd(const Kv8Tc& p, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (!p.kx) return launch_variant<HD, true, T>(p, s);
  return launch_variant<HD, false, T>(p, s);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

void reset_kv8_tc_caches() {
  std::lock_guard<std::mutex> g(g_tc_mu);
  for (auto& dev : g_tc)
    for (auto& d : dev) d = TcDevice{};
}

// Which calls take this path: head_dim 64 or 128, and enough query rows per KV head.  Its
// time hardly depends on the rows (up to a tile), the other's grows with every 8 of them.
// 24 / 32 / 40 rows, hd 128, other's times and this one's: 32 heads over 4096 keys 33, 38, 41 and
// 24 us; 8 over 16384 32, 35, 42 and 39 us; 8 sequences of 8 over 8192 61, 73, 87 and 71 us.  With
// the weights, 16 / 24 rows: 46, 61 and 41 us; 48, 59 and 56 us; 115, 141 and 124 us.  fp32, 32 / 48 /
// 96 rows: 32 heads over 4096 keys 43, 54, 88 and 42 us; 8 over 16384 40, 54, 89 and 52 us; 4 sequences
// of 4 over 8192 34, 43, 69 and 54 us; with the weights, 16 / 24 rows: 62, 86 and 58 us; 65, 85 and 68
// us; 59, 71 and 68 us.  The rule goes by rows alone; where the (sequence, KV head) units are few
// and the rows just past the bound the other path would still be faster, by a quarter at the most
// (8 heads over 16384 keys at 32 rows 35 and 39 us, fp32 4 x 4 over 8192 at 49 rows 43 and 54).
bool kv8_tc_taken(int dt, int hd, int G, int n_q, bool weights) {
  return (hd == 64 || hd == 128) && G <= BM && (int64_t)n_q * G > (weights ? 16 : dt == DT_F32 ? 48 : 24) &&
         (n_q + BM / G - 1) / (BM / G) <= 65535;
}

// One query tile: the codes are converted where they are used (fp32's two parts of q leave no room
// for them).  With two tiles it gains in few shapes and loses in most: 200 rows of 32 heads over
// 4096 keys 41 us instead of 45, but 250 of 40 over 8192 116 instead of 110, 140 of 4 over 16384 39
// instead of 34, with weights 50 instead of 44.
static bool is_fused(int dt, int G, int n_q) { return dt == DT_BF16 && n_q <= BM / G; }
bool kv8_tc_expands(int dt, int G, int n_q) { return !is_fused(dt, G, n_q); }

namespace {
struct WsOff {
  size_t vx, seq_max, qx, rows, tile_max, bytes;
};
WsOff ws_of(int dt, int n_seq, int Hkv, int G, int n_q, int64_t cap, int hd, bool weights) {
  const size_t tile = (size_t)BN * hd * 2, kt = (size_t)n_seq * Hkv * ((cap + BN - 1) / BN);
  const size_t qt = (n_q + BM / G - 1) / (BM / G), all = (size_t)n_seq * Hkv * qt;
  WsOff w{};
  if (!is_fused(dt, G, n_q)) {
    w.vx = align256(kt * tile);
    w.seq_max = w.vx + align256(kt * tile);
    w.qx = w.seq_max + align256((size_t)n_seq * 4);
  }
  const int np = dt == DT_F32 ? 2 : 1;
  w.rows = w.qx + (weights ? align256(all * tile * np) : 0);
  w.tile_max = w.rows + (weights ? align256(all * (np + 1) * BM * 4) : 0);
  w.bytes = w.tile_max + (weights ? align256((size_t)n_seq * qt * 4) : 0);
  return w;
}
}  // namespace

// (the operands are written in 32-byte words: room to start on a boundary of those)
size_t kv8_tc_ws_bytes(int dt, int n_seq, int Hkv, int G, int n_q, int64_t cap, int hd, bool weights) {
  const size_t n = ws_of(dt, n_seq, Hkv, G, n_q, cap, hd, weights).bytes;
  return n ? n + 32 : 0;
}

cudaError_t launch_kv8_tc(int dt, const void* q, const int32_t* last, int n_q, const cb_kv8_cache& c, int H, int Hkv, int hd,
                          void* out, float* weights, void* ws, cudaStream_t s) {
  g_used_kv8_tc = true;
  Kv8Tc p{};
  p.q = q;
  p.last = last;
  p.out = out;
  p.c = c;
  p.n_q = n_q;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.lg = 31 - __builtin_clz((unsigned)c.block);
  p.tiles = (int)((c.capacity + BN - 1) / BN);
  p.qpt = BM / p.G;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)hd);
  p.q_tiles = (n_q + p.qpt - 1) / p.qpt;
  p.g_magic = ((1 << 16) + p.G - 1) / p.G;
  const WsOff w = ws_of(dt, c.n_seq, Hkv, p.G, n_q, c.capacity, hd, weights != nullptr);
  uint8_t* b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31));
  if (!is_fused(dt, p.G, n_q)) {
    p.kx = b;
    p.vx = b + w.vx;
    p.seq_max = reinterpret_cast<int32_t*>(b + w.seq_max);
  }
  if (weights) {
    p.qx = b + w.qx;
    p.rows = reinterpret_cast<float*>(b + w.rows);
    p.tile_max = reinterpret_cast<int32_t*>(b + w.tile_max);
    if (!p.seq_max) p.seq_max = p.tile_max;      // one tile per sequence
    p.weights = weights;
  }
  if (dt == DT_F32) return hd == 128 ? launch_hd<128, float>(p, s) : launch_hd<64, float>(p, s);
  return hd == 128 ? launch_hd<128, bf16>(p, s) : launch_hd<64, bf16>(p, s);
}

}  // namespace cb
