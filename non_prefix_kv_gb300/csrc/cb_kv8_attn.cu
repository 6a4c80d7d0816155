// Attention over the 8-bit block-scaled KV cache (cb_kv8.cu), for a few query rows per KV head
// (single tokens) and, in tiles of 8 rows, for any number.
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
// the rounding of the bf16 output (2^-8), for fp32 output split in two parts.  bf16 rows take
// log2 vs and 1 / vs by the approximate instructions, each off by 2 ulp: of log2 vs, which goes into
// the exponent, that is 2^-20 at vs = 0.03 and 2^-18 at the smallest scale, still below fp16's 2^-11;
// fp32 rows take log2f.  Sums, maxima and accumulators are fp32.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "cb_kv8.cuh"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_kv8_attn;
static std::atomic<bool> g_used_kv8_attn{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_kv8_attn() { return g_used_kv8_attn ? take_word(g_err_kv8_attn) : 0u; }

namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr float kPBias = 8.0f;       // 2^(t - m) is held up to 2^8 ...
constexpr float kLazy = 6.0f;        // ... and up to 2^14 before m is raised: fp16 ends at 2^16
constexpr float kNone = -1e30f;      // m of a row that has seen no key
constexpr float kMinFactor = 1.17549435e-38f;   // a score's factor is no smaller: times an unseen score of -inf, 0 is NaN
constexpr int TILE = 8;              // query rows of a tile
constexpr int MAX_WORKERS = 4096;    // warps of the largest grid (a workspace is sized without the device)

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
using tc::bulk_load;

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
  int32_t* plan;            // [entries + 1] steps before each (sequence, row tile), times Hkv
  float* part;              // partial results, see slot()
  float* z;                 // [n_seq * Hkv, n_q * G, capacity] scores z_i for the weights, or null
  float* lse;               // [n_seq * Hkv, n_q * G] log2 of a row's sum for k_kv8_weights, or null
  float* weights;           // [n_seq, Hkv, capacity], or null
  cb_kv8_cache c;
  int n_q, H, Hkv, G, lg;
  int row_tiles;            // tiles of a sequence's query rows
  float scale_log2;         // log2(e) / sqrt(hd)
};

// A step is 16 KW keys: 4 KB of codes (8 KB at head_dim 256).  Each warp keeps three of them in
// flight in its own shared memory: with 16 warps per SM (8 at 256) 192 KB of loads.
template <int HD>
struct Lay {
  static constexpr int KW = HD < 128 ? 128 / HD : 1;               // groups of 16 keys per step
  static constexpr int KT = 16 * KW;
  static constexpr int HALF = KT * HD;                             // K (or V) codes of a step
  static constexpr int NST = 3;
  static constexpr int OFF_BAR = WARPS * NST * 2 * HALF;           // [WARPS][NST]
  static constexpr int OFF_SUM = OFF_BAR + WARPS * NST * 8;        // [THREADS] steps before a thread's entries
  static constexpr int BYTES = OFF_SUM + THREADS * 4 + 128;
};
// fp16 parts of q and of the weights
template <typename T>
constexpr int parts() {
  return sizeof(T) == 4 ? 2 : 1;
}
template <int HD, typename T>
constexpr int ctas_per_sm() {
  return HD == 256 ? 1 : 2;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, bool on, float* f) {
  if (on) {
    ld4(p, f);
  } else {
    f[0] = f[1] = f[2] = f[3] = 0.f;
  }
}

// The last cache row that query j of sequence s sees; -1 where its bound is bad (reported if asked).
__device__ __forceinline__ int query_last(const Kv8Attn& p, int s, int j, bool report) {
  const int l = p.last[(int64_t)s * p.n_q + j];
  if (l < -1 || l >= p.c.capacity) {
    if (report) atomicOr(&g_err_kv8_attn, ERRBIT_INDEX);
    return -1;
  }
  return l;
}
// The same for row r of entry e (sequence e / row_tiles, row tile e % row_tiles), -1 where the row
// does not exist.
__device__ __forceinline__ int row_last(const Kv8Attn& p, int e, int r) {
  const int s = e / p.row_tiles, row = (e - s * p.row_tiles) * TILE + r;
  return r >= TILE || row >= p.n_q * p.G ? -1 : query_last(p, s, row / p.G, false);
}

// The line of work: unit (entry e, KV head h) holds the steps of the entry's visible keys;
// units follow one another by entry, then head, and the line is cut into equal runs, one per
// worker (a warp).  A run may end inside a unit and hold several; each (worker, unit) pair
// leaves one partial result.  Along the line either the worker or the unit goes up at every
// new pair, so worker + unit numbers the pairs' slots without a gap wider than one.  A run has two
// steps at least (a token of 32 heads over 512 / 2048 rows: 11.8 and 13.1 us; with one step 11.0 and
// 14.0, with four 12.1 and 13.8, with eight 15.0 and 17.3).
__device__ __forceinline__ int workers_of(int total, int workers) { return max(1, min(workers, total / 2)); }
// the first step of worker w's run: floor(total w / n), w <= n <= 2^12, without a 64-bit division
__device__ __forceinline__ int run_start(int total, int w, int n) {
  const unsigned each = (unsigned)total / (unsigned)n, rest = (unsigned)total - each * n;
  return (int)(each * w + rest * w / n);
}
// the worker whose run holds step x: floor(((x + 1) n - 1) / total) (run_start(w + 1) > x says
// (w + 1) total >= (x + 1) n); the fp32 quotient is off by less than one
__device__ __forceinline__ int worker_of(int total, int x, int n) {
  const int64_t a = ((int64_t)x + 1) * n - 1;
  int w = (int)__fdividef((float)a, (float)total);
  if ((int64_t)w * total > a) --w;
  if ((int64_t)(w + 1) * total <= a) ++w;
  return w;
}
__device__ __forceinline__ float* slot(const Kv8Attn& p, int hd, int worker, int unit) {
  const int rows = min(TILE, p.n_q * p.G);
  return p.part + ((int64_t)worker + unit) * (rows * hd + 2 * TILE);     // [rt] max, [rt] sum, [rows][hd] O
}

// Single tokens are bound by the cache's bytes, and a grid of CTAs per (sequence, head) leaves
// a third of them on the table: with 32 sequences of 9000..16384 rows and 8 heads (841 MB) it
// took 167 us, though one full wave of equal CTAs ran at 0.96 of the copy rate (whole waves,
// lengths that differ, and about 10 us of start, fill and merge per CTA).  So every warp of a
// grid that fills the machine once takes an equal run of the line above, streams it through its
// own stages, and meets no other warp; k_kv8_merge joins the partial results.
//
// The products are taken transposed, S^T = C_K Q^T and O^T = C_V^T P^T, with the keys (then the
// channels) as the 16 rows of mma.m16n8k16 and the query rows as its 8 columns: the few rows of
// a token fill the instruction, and a thread's share of O is HD / 4 registers, so that 16
// warps fit on an SM.  (With rows as M and 10 warps: 205 us at an issue rate of 0.33; with two row
// tiles per instruction stream where there are more than 8 rows, 32 rows of 32 heads over 4096
// keys 48 us instead of 38.)  Now 144 us for the 841 MB, 5.85 TB/s, merge included; bound by the
// bytes and, at a busy issue slot in two cycles, by the conversion of the codes.  One token of 32
// heads over 4096 rows (34 MB): 11.3 us and 4.6 more for the merge, bound by start and latency.
template <int HD, typename T>
__global__ void __launch_bounds__(THREADS, ctas_per_sm<HD, T>()) k_kv8_attn(const Kv8Attn p) {
  pdl_wait();
  pdl_trigger();
  using L = Lay<HD>;
  constexpr int NS = parts<T>();
  constexpr int KS = HD / 16;                    // k steps of a score; also channel tiles of O
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((128 - (tc::smem_u32(smem_raw) & 127)) & 127);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* stages = base + warp * L::NST * 2 * L::HALF;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + L::OFF_BAR) + warp * L::NST;
  int* before = reinterpret_cast<int*>(base + L::OFF_SUM);
  const int R = p.n_q * p.G, entries = p.c.n_seq * p.row_tiles;
  const int64_t cap = p.c.capacity;
  if (lane == 0)
    for (int i = 0; i < L::NST; ++i) tc::mbar_init(&full[i], 1);
  if (lane == 0) tc::fence_mbar_init();

  // ---- where this worker's run lies: thread i sums the steps of a contiguous share of the
  // entries, a scan over the threads places them (the first CTA writes the plan for the merge)
  auto steps_of = [&](int e, bool report) -> int {
    const int s = e / p.row_tiles, row0 = (e - s * p.row_tiles) * TILE;
    int mx = -1;
    for (int j = row0 / p.G; j <= (min(R, row0 + TILE) - 1) / p.G; ++j) mx = max(mx, query_last(p, s, j, report));
    return (mx + L::KT) / L::KT;
  };
  const int share = (entries + THREADS - 1) / THREADS, e0 = min(entries, tid * share), e1 = min(entries, e0 + share);
  int own = 0;
  for (int e = e0; e < e1; ++e) own += steps_of(e, blockIdx.x == 0) * p.Hkv;
  int incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __shared__ int wsum[WARPS];
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) incl += wsum[w];
    total += wsum[w];
  }
  before[tid] = incl - own;
  if (blockIdx.x == 0) {
    int at = incl - own;
    for (int e = e0; e < e1; ++e) {
      p.plan[e] = at;
      at += steps_of(e, false) * p.Hkv;
    }
    if (tid == 0) p.plan[entries] = total;
  }
  __syncthreads();
  // consecutive workers sit in different CTAs, so that few of them still spread over the SMs
  const int n_work = workers_of(total, gridDim.x * WARPS), worker = warp * gridDim.x + blockIdx.x;
  if (worker >= n_work) return;                  // no barrier of the CTA follows
  const int a = run_start(total, worker, n_work), b = run_start(total, worker + 1, n_work);
  if (a >= b) return;

  // steps of entry e, by the whole warp
  auto warp_steps = [&](int e) -> int {
    return (__reduce_max_sync(0xffffffffu, row_last(p, e, lane)) + L::KT) / L::KT;
  };
  struct Pos {
    int e, h, k, n;       // entry, head, step of the unit, steps in a unit of the entry
  };
  auto to_entry = [&](Pos& x) {                  // skips entries without a step; stops at the last
    while (x.e < entries && (x.n = warp_steps(x.e)) == 0) ++x.e;
  };
  auto advance = [&](Pos& x) {
    if (++x.k < x.n) return;
    x.k = 0;
    if (++x.h < p.Hkv) return;
    x.h = 0;
    ++x.e;
    to_entry(x);
  };
  Pos cur;
  {
    // the last thread whose share starts at or before the run
    int c = 0;
    for (int i = lane; i < THREADS; i += 32)
      if (before[i] <= a && i * share < entries) c = i;
    c = __reduce_max_sync(0xffffffffu, c);
    cur.e = c * share;
    int left = a - before[c];
    for (;; ++cur.e) {
      cur.n = warp_steps(cur.e);
      if (left < cur.n * p.Hkv) break;
      left -= cur.n * p.Hkv;
    }
    cur.h = left / cur.n;
    cur.k = left - cur.h * cur.n;
  }
  auto fill = [&](const Pos& x, int st) {
    if (lane != 0) return;
    const int64_t k0 = (int64_t)x.k * L::KT, at = (((int64_t)(x.e / p.row_tiles) * p.Hkv + x.h) * cap + k0) * HD;
    const uint32_t bytes = (uint32_t)(cap - k0 < L::KT ? cap - k0 : L::KT) * HD;
    tc::mbar_expect_tx(&full[st], 2 * bytes);
    bulk_load(stages + st * 2 * L::HALF, p.c.k_codes + at, bytes, &full[st]);
    bulk_load(stages + st * 2 * L::HALF + L::HALF, p.c.v_codes + at, bytes, &full[st]);
  };
  Pos pre = cur;                                 // the next step to load
  int loaded = 0;
  for (; loaded < L::NST && a + loaded < b; ++loaded) {
    fill(pre, loaded);
    if (a + loaded + 1 < b) advance(pre);
  }

  bool ok = true;
  for (int i = a; ok && i < b;) {
    // ------------------------------------------------------------------ a unit, or a part of one
    const int s = cur.e / p.row_tiles, row0 = (cur.e - s * p.row_tiles) * TILE, nrow = min(TILE, R - row0), h = cur.h;
    const int64_t head = (int64_t)s * p.Hkv + h;
    const int my_last = row_last(p, cur.e, lane);
    const int nk = __reduce_max_sync(0xffffffffu, my_last) + 1;       // keys some row sees
    const int mn = __reduce_min_sync(0xffffffffu, lane < nrow ? my_last : 0x7fffffff);
    const float* ksc = p.c.k_scale + head * (cap >> p.lg);
    const float* vsc = p.c.v_scale + head * (cap >> p.lg);
    // scales of the next 16 keys, loaded one group ahead (1 past the visible keys: their block
    // may never have been written)
    auto scales_of = [&](int key) -> float2 {
      float2 r = make_float2(1.0f, 1.0f);
      if (key < nk) {
        r.x = ksc[key >> p.lg];
        r.y = vsc[key >> p.lg];
      }
      return r;
    };
    float2 next = scales_of(cur.k * L::KT);
    // Q^T as the column operand: thread (g, t) holds row g, channels [t HD/4, (t + 1) HD/4),
    // 4 per k step (the order of the channels inside a sum is free; K is read with the same one)
    uint2 qb[NS][KS];
    float rf[2];                             // score factor of rows 2t, 2t + 1
    int lastr[2];
    const int r = row0 + g;
    const bool on = g < nrow;
    const int j = on ? r / p.G : 0;
    const T* qr = static_cast<const T*>(p.q) +
                  (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (on ? r - j * p.G : 0)) * HD + t * (HD / 4);
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      float f[4];
      load4(qr + 4 * ks, on, f);
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^ex <= amax < 2^(ex + 1); both powers stay normal
    int ex = amax > 0.f ? ilogbf(amax) : 0;
    ex = ex < -120 ? -120 : (ex > 120 ? 120 : ex);
    const float down = ldexpf(1.0f, -ex), up = ldexpf(p.scale_log2, ex);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      float f[4];
      load4(qr + 4 * ks, on, f);
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] *= down;
      qb[0][ks] = make_uint2(pack_h2(f[0], f[1]), pack_h2(f[2], f[3]));
      if constexpr (NS == 2)
        qb[1][ks] = make_uint2(rest_h2(f[0], f[1], qb[0][ks].x), rest_h2(f[2], f[3], qb[0][ks].y));
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      rf[c] = __shfl_sync(0xffffffffu, up, (2 * t + c) * 4);
      lastr[c] = __shfl_sync(0xffffffffu, my_last, 2 * t + c);
    }
    float* z = p.z ? p.z + (head * R + row0) * cap : nullptr;
    float O[KS][4];                          // channel tile: rows 2t, 2t + 1 of channels g, g + 8
    float m_used[2], l_sum[2];           // of rows 2t, 2t + 1 (l: this thread's keys)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m_used[c] = kNone;
      l_sum[c] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) O[k][c] = 0.f;
    const int end = min(b, i + cur.n - cur.k);   // line position after this unit's share
    const int unit = cur.e * p.Hkv + h;
    int k0 = cur.k * L::KT;
    for (; i < end; ++i, k0 += L::KT) {
      const int u = i - a, st = u % L::NST;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[st], (u / L::NST) & 1));
      if (!ok) break;
      const uint8_t* sk = stages + st * 2 * L::HALF;
#pragma unroll 1
      for (int w = 0; w < L::KW; ++w) {
        const int key0 = k0 + w * 16;
        const float2 now = next;
        next = scales_of(key0 + 16);
        if (key0 >= nk) continue;
        // ---- scores of 16 keys: thread (g, t) reads keys g and g + 8
        float S[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) S[c] = 0.f;
        const uint8_t* kr = sk + (w * 16 + g) * HD + t * (HD / 4);
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
          for (int q = 0; q < KC / 4; ++q) {
            const int ks = c0 / 4 + q;
            uint32_t x[4];                                    // rows g, g + 8 of channels 4 ks .. + 1, then + 2 .. + 3
            codes_to_h2(w0[q], x[0], x[2]);
            codes_to_h2(w1[q], x[1], x[3]);
#pragma unroll
            for (int part = 0; part < NS; ++part) mma_f16(S, x, qb[part][ks].x, qb[part][ks].y);
          }
        }
        // ---- weights: element c of S is key g + 8 (c / 2), row 2t + c % 2
        const float vs = fmaxf(now.y, kKv8MinScale);
        const float3 sc = make_float3(fmaxf(now.x, kKv8MinScale), NS == 2 ? log2f(vs) : __log2f(vs), __fdividef(1.0f, vs));
        const bool whole = key0 + 15 <= mn;                   // every row sees every key
        float f[2], add[2], ev[4];
        bool high = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          f[c] = fmaxf(rf[c] * sc.x, kMinFactor);             // (below it no score reaches 2^-100)
          add[c] = sc.y - m_used[c] + kPBias;
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (key0 + g + 8 * (c >> 1) > lastr[c & 1]) S[c] = -INFINITY;
        }
        if (z) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (2 * t + (c & 1) < nrow)
              z[(2 * t + (c & 1)) * cap + key0 + g + 8 * (c >> 1)] = S[c] * f[c & 1];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) ev[c] = fmaf(S[c], f[c & 1], add[c & 1]);
        high |= fmaxf(fmaxf(ev[0], ev[1]), fmaxf(ev[2], ev[3])) > kPBias + kLazy;
        // m is raised when a weight would leave fp16's range (and at a row's first key)
        if (__any_sync(0xffffffffu, high)) {
          float al[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float tt = fmaxf(S[c], S[c + 2]) * f[c];
            tt = fmaxf(tt, __shfl_xor_sync(0xffffffffu, tt, 4));
            tt = fmaxf(tt, __shfl_xor_sync(0xffffffffu, tt, 8));
            tt = fmaxf(tt, __shfl_xor_sync(0xffffffffu, tt, 16)) + sc.y;
            const bool raise = tt > m_used[c] + kLazy;
            al[c] = raise ? tc::ex2_approx(m_used[c] - tt) : 1.0f;
            if (raise) m_used[c] = tt;
            l_sum[c] *= al[c];
            add[c] = sc.y - m_used[c] + kPBias;
            ev[c] = fmaf(S[c], f[c], add[c]);
            ev[c + 2] = fmaf(S[c + 2], f[c], add[c]);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) O[k][c] *= al[c & 1];
        }
        uint32_t pb[NS][2];
#pragma unroll
        for (int c = 0; c < 4; ++c) ev[c] = tc::ex2_approx(ev[c]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = pack_h2(ev[2 * k], ev[2 * k + 1]);
          pb[0][k] = transpose_h2(x);
          if constexpr (NS == 2) pb[1][k] = transpose_h2(rest_h2(ev[2 * k], ev[2 * k + 1], x));
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) l_sum[c] = fmaf(ev[c] + ev[c + 2], sc.z, l_sum[c]);
        // ---- O^T += C_V^T P^T: this thread's V rows are keys 2t, 2t+1, 2t+8, 2t+9; rows g, g + 8
        // of channel tile k stand for channels (HD/8) g + 2 k, + 1
        const uint8_t* vr = sk + L::HALF + (w * 16 + 2 * t) * HD + g * (HD / 8);
        constexpr int VC = HD >= 128 ? 16 : HD / 8;           // bytes per load
#pragma unroll
        for (int c0 = 0; c0 < HD / 8; c0 += VC) {
          uint32_t v[4][VC / 4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint8_t* at = vr + ((r & 1) + 8 * (r >> 1)) * HD + c0;
            if constexpr (VC == 16) {
              const uint4 x = *reinterpret_cast<const uint4*>(at);
              v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
            } else if constexpr (VC == 8) {
              const uint2 x = *reinterpret_cast<const uint2*>(at);
              v[r][0] = x.x; v[r][1] = x.y;
            } else {
              v[r][0] = *reinterpret_cast<const uint32_t*>(at);
            }
          }
#pragma unroll
          for (int c = 0; c < VC / 4; ++c) {
            const uint32_t x0[4] = {codes_pair<0>(v[0][c], v[1][c]), codes_pair<1>(v[0][c], v[1][c]),
                                    codes_pair<0>(v[2][c], v[3][c]), codes_pair<1>(v[2][c], v[3][c])};
            const uint32_t x1[4] = {codes_pair<2>(v[0][c], v[1][c]), codes_pair<3>(v[0][c], v[1][c]),
                                    codes_pair<2>(v[2][c], v[3][c]), codes_pair<3>(v[2][c], v[3][c])};
            const int k = c0 / 2 + 2 * c;
#pragma unroll
            for (int part = 0; part < NS; ++part) {
              mma_f16(O[k], x0, pb[part][0], pb[part][1]);
              mma_f16(O[k + 1], x1, pb[part][0], pb[part][1]);
            }
          }
        }
      }
      __syncwarp();                              // every lane has read the stage: refill it
      if (a + loaded < b) {
        fill(pre, st);
        ++loaded;
        if (a + loaded < b) advance(pre);
      }
    }
    if (!ok) break;
    // ------------------------------------------------------------------ the partial result
    float* dst = slot(p, HD, worker, unit);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 2 * t + c;
      float l = l_sum[c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {
        dst[r] = m_used[c];
        dst[TILE + r] = l;
      }
      if (r < nrow) {
        float* o = dst + 2 * TILE + r * HD + (HD / 8) * g;
#pragma unroll
        for (int k = 0; k < KS; k += 2)
          *reinterpret_cast<float4*>(o + 2 * k) = make_float4(O[k][c], O[k][c + 2], O[k + 1][c], O[k + 1][c + 2]);
      }
    }
    cur.k = 0;
    if (i < b) {                                 // the run goes on: the unit was finished
      if (++cur.h == p.Hkv) {
        cur.h = 0;
        ++cur.e;
        to_entry(cur);
      }
    }
  }
  if (!ok) {
    // report, and give the copies in flight as long again before the memory is given up
    if (lane == 0) atomicOr(&g_err_kv8_attn, ERRBIT_TIMEOUT);
    for (int k = loaded > L::NST ? loaded - L::NST : 0; k < loaded; ++k) tc::mbar_wait(&full[k % L::NST], (k / L::NST) & 1);
  }
}

// The workers whose runs meet unit (entry e, head h): the first one, and how many.
__device__ __forceinline__ int unit_workers(const Kv8Attn& p, int e, int h, int max_workers, int* first) {
  const int start = p.plan[e], n = (p.plan[e + 1] - start) / p.Hkv, total = p.plan[p.c.n_seq * p.row_tiles];
  if (n <= 0) return 0;
  const int nw = workers_of(total, max_workers), x0 = start + h * n;
  *first = worker_of(total, x0, nw);
  return worker_of(total, x0 + n - 1, nw) - *first + 1;
}

// The account of the weights, one row tile: weights[key] += sum over the rows of 2^(z - log2 of the
// row's sum), four keys per thread.  A CTA takes a (sequence, head)'s next 1024 keys and joins the
// rows' sums itself, a warp per row, so that it need not wait for the merge: it is launched with it
// (a token with weights, 32 heads over 1024 rows: 10.4 us, 13.8 as a launch of its own).
__device__ __forceinline__ void account(const Kv8Attn& p, int hd, int block, int max_workers) {
  __shared__ float s_lse[TILE];
  const int64_t cap = p.c.capacity;
  const int chunks = (int)((cap + 1023) / 1024), head = block / chunks, s = head / p.Hkv, h = head - s * p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = p.n_q * p.G;
  const int64_t key = ((int64_t)(block - head * chunks) * 256 + threadIdx.x) * 4;
  int mx = -1;
  for (int r = 0; r < R; r += p.G) mx = max(mx, query_last(p, s, r / p.G, false));
  if (key - threadIdx.x * 4 > mx) return;          // whole CTAs
  if (warp < R) {
    int w0 = 0;
    const int np = unit_workers(p, s, h, max_workers, &w0);
    float mm = kNone, sum = 0.f;
    for (int i = lane; i < np + lane; i += 32) {   // whole warps
      float m = kNone, l = 0.f;
      if (i < np) {
        const float* src = slot(p, hd, w0 + i, head);
        m = src[warp];
        l = src[TILE + warp];
      }
      const float top = fmaxf(mm, warp_max(m));
      sum = fmaf(sum, tc::ex2_approx(mm - top), warp_sum(l * tc::ex2_approx(m - top)));
      mm = top;
    }
    if (lane == 0) s_lse[warp] = sum == 0.f ? INFINITY : mm - kPBias + log2f(sum);
  }
  __syncthreads();
  if (key > mx) return;
  const float* z = p.z + head * R * cap + key;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r = 0; r < R; ++r) {
    const float4 v = *reinterpret_cast<const float4*>(z + r * cap);     // an unseen key's z is -inf
    const float l = s_lse[r];
    a[0] += v.x == -INFINITY ? 0.f : tc::ex2_approx(v.x - l);           // (l of a NaN query is NaN)
    a[1] += v.y == -INFINITY ? 0.f : tc::ex2_approx(v.y - l);
    a[2] += v.z == -INFINITY ? 0.f : tc::ex2_approx(v.z - l);
    a[3] += v.w == -INFINITY ? 0.f : tc::ex2_approx(v.w - l);
  }
  float* w = p.weights + (int64_t)head * cap + key;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (key + k <= mx) w[k] += a[k];
}

// Joins the partial results of one query row: the workers whose runs meet its unit, their
// maxima and sums, then the weighted sum of their O.  WPR warps per (row, unit), each taking
// every WPR-th worker, 32 at a time (a lane per worker for the statistics, a lane per HD / 32
// channels for O); with several warps their results meet in shared memory.
constexpr int MERGE_WARPS = 8;
template <int HD, int WPR, typename T>
__global__ void __launch_bounds__(32 * MERGE_WARPS) k_kv8_merge(const Kv8Attn p, int max_workers, int merge_ctas) {
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= merge_ctas) {             // CTAs past the merge's: the account
    account(p, HD, blockIdx.x - merge_ctas, max_workers);
    return;
  }
  constexpr int PL = HD / 32;          // channels of a lane
  __shared__ float s_o[WPR > 1 ? MERGE_WARPS : 1][HD];
  __shared__ float s_m[MERGE_WARPS], s_l[MERGE_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int rows = min(TILE, p.n_q * p.G), entries = p.c.n_seq * p.row_tiles;
  const int item = blockIdx.x * (MERGE_WARPS / WPR) + warp / WPR;    // (entry, head, row of the tile)
  if (item >= entries * p.Hkv * rows) return;    // whole CTAs when WPR = MERGE_WARPS
  const int unit = item / rows, r = item - unit * rows, e = unit / p.Hkv, h = unit - e * p.Hkv;
  const int s = e / p.row_tiles, row = (e - s * p.row_tiles) * TILE + r, R = p.n_q * p.G;
  int w0 = 0;
  const int np = row < R ? unit_workers(p, e, h, max_workers, &w0) : 0;
  float mm = kNone, sum = 0.f, o[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) o[k] = 0.f;
  for (int i0 = sub; i0 < np; i0 += 32 * WPR) {
    const int mine = i0 + lane * WPR;
    float m = kNone, l = 0.f;
    if (mine < np) {
      const float* src = slot(p, HD, w0 + mine, unit);
      m = src[r];
      l = src[TILE + r];
    }
    const float top = fmaxf(mm, warp_max(m)), back = tc::ex2_approx(mm - top), f = tc::ex2_approx(m - top);
    mm = top;
    sum = fmaf(sum, back, warp_sum(l * f));
#pragma unroll
    for (int k = 0; k < PL; ++k) o[k] *= back;
    const int cnt = min(32, (np - i0 + WPR - 1) / WPR);
#pragma unroll 8
    for (int i = 0; i < cnt; ++i) {
      const float* src = slot(p, HD, w0 + i0 + i * WPR, unit) + 2 * TILE + r * HD + lane * PL;
      const float fi = __shfl_sync(0xffffffffu, f, i);
      float v[PL];
      if constexpr (PL >= 4) {
#pragma unroll
        for (int k = 0; k < PL; k += 4) ld4(src + k, v + k);
      } else if constexpr (PL == 2) {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] = x.x;
        v[1] = x.y;
      } else {
        v[0] = *src;
      }
#pragma unroll
      for (int k = 0; k < PL; ++k) o[k] = fmaf(v[k], fi, o[k]);
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      s_m[warp] = mm;
      s_l[warp] = sum;
    }
#pragma unroll
    for (int k = 0; k < PL; ++k) s_o[warp][lane * PL + k] = o[k];
    __syncthreads();
    if (sub != 0) return;
    float top = mm;
#pragma unroll
    for (int w = 1; w < WPR; ++w) top = fmaxf(top, s_m[w]);
    const float f0 = tc::ex2_approx(mm - top);
    sum *= f0;
#pragma unroll
    for (int k = 0; k < PL; ++k) o[k] *= f0;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      const float f = tc::ex2_approx(s_m[w] - top);
      sum = fmaf(s_l[w], f, sum);
#pragma unroll
      for (int k = 0; k < PL; ++k) o[k] = fmaf(s_o[w][lane * PL + k], f, o[k]);
    }
    mm = top;
  }
  if (row >= R) return;
  // a row that sees nothing is 0 and weighs nothing; a NaN stays one
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
  const int64_t head = (int64_t)s * p.Hkv + h;
  if (p.lse && lane == 0) p.lse[head * R + row] = sum == 0.f ? INFINITY : mm - kPBias + log2f(sum);
  const int j = row / p.G;
  T* out = static_cast<T*>(p.out) + (((int64_t)s * p.n_q + j) * p.H + (int64_t)h * p.G + (row - j * p.G)) * HD + lane * PL;
#pragma unroll
  for (int k = 0; k < PL; ++k) o[k] *= inv;
  if constexpr (PL >= 4) {
#pragma unroll
    for (int k = 0; k < PL; k += 4) st4(out + k, o + k);
  } else {
#pragma unroll
    for (int k = 0; k < PL; ++k) out[k] = from_f<T>(o[k]);
  }
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

template <int HD, typename T>
cudaError_t prepare_attn(int dev) {
  constexpr int h = HD == 32 ? 0 : HD == 64 ? 1 : HD == 128 ? 2 : 3;
  constexpr uint32_t bit = 1u << (h + (sizeof(T) == 4 ? 4 : 0));
  std::lock_guard<std::mutex> g(g_kv8_mu);
  if (dev >= 0 && dev < 64 && (g_kv8_attr[dev] & bit)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<HD>::BYTES);
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
  const int ctas = std::min(ctas_per_sm<HD, T>() * device_sms(dev), MAX_WORKERS / WARPS);
  if ((e = launch_k(k_kv8_attn<HD, T>, dim3(ctas), dim3(THREADS), Lay<HD>::BYTES, s, p)) != cudaSuccess) return e;
  const int64_t items = (int64_t)p.c.n_seq * p.row_tiles * p.Hkv * std::min(TILE, p.n_q * p.G);
  // a warp per row where that alone fills the SMs, else a CTA (32 sequences of 8 x 7 heads, 1792
  // rows whose units meet 10 workers each: 144 and 148 us; one of 32 heads, 32 rows and 75
  // workers: 28 and 17 us; 8 of 32 heads, 256 rows and 10 workers: 48 and 46 us)
  const int64_t acc = p.z ? (p.c.capacity + 1023) / 1024 * p.Hkv * p.c.n_seq : 0;
  if (items >= (int64_t)MERGE_WARPS * device_sms(dev)) {
    const int n = (int)((items + MERGE_WARPS - 1) / MERGE_WARPS);
    return launch_k(k_kv8_merge<HD, 1, T>, dim3((unsigned)(n + acc)), dim3(32 * MERGE_WARPS), 0, s, p, ctas * WARPS, n);
  }
  return launch_k(k_kv8_merge<HD, MERGE_WARPS, T>, dim3((unsigned)(items + acc)), dim3(32 * MERGE_WARPS), 0, s, p,
                  ctas * WARPS, (int)items);
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

// whether the weights of several row tiles are taken by a kernel of their own, from the row sums
bool kv8_attn_weights_apart(int G, int n_q) { return (int64_t)n_q * G > TILE; }

namespace {
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
// the workspace: plan, partial results, and for the weights the row sums and (one tile) the scores
struct WsOff {
  size_t part, lse, z, bytes;
};
WsOff ws_of(int n_seq, int Hkv, int G, int n_q, int64_t cap, int hd, bool weights) {
  const size_t R = (size_t)n_q * G, tiles = (R + TILE - 1) / TILE;
  WsOff w;
  w.part = up256(((size_t)n_seq * tiles + 1) * 4);
  w.lse = w.part + up256(((size_t)n_seq * tiles * Hkv + MAX_WORKERS) * (std::min((size_t)TILE, R) * hd + 2 * TILE) * 4);
  const bool apart = kv8_attn_weights_apart(G, n_q);
  w.z = w.lse + (weights && apart ? up256((size_t)n_seq * Hkv * R * 4) : 0);
  w.bytes = w.z + (weights && !apart ? (size_t)n_seq * Hkv * R * cap * 4 : 0);
  return w;
}
}  // namespace

size_t kv8_attn_ws_bytes(int n_seq, int Hkv, int G, int n_q, int64_t cap, int hd, bool weights) {
  return ws_of(n_seq, Hkv, G, n_q, cap, hd, weights).bytes;
}

static Kv8Attn make_params(const void* q, const int32_t* last, int n_q, const cb_kv8_cache& c, int H, int Hkv,
                           int hd, void* out, float* weights, void* ws) {
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
  const int64_t R = (int64_t)n_q * p.G;
  p.row_tiles = (int)((R + TILE - 1) / TILE);
  const WsOff w = ws_of(c.n_seq, Hkv, p.G, n_q, c.capacity, hd, weights != nullptr);
  char* b = static_cast<char*>(ws);
  p.plan = reinterpret_cast<int32_t*>(b);
  p.part = reinterpret_cast<float*>(b + w.part);
  if (weights) {
    p.weights = weights;
    if (kv8_attn_weights_apart(p.G, n_q))
      p.lse = reinterpret_cast<float*>(b + w.lse);
    else
      p.z = reinterpret_cast<float*>(b + w.z);
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
  g_used_kv8_attn = true;
  const Kv8Attn p = make_params(q, last, n_q, c, H, Hkv, hd, out, weights, ws);
  CB_KV8_DISPATCH(launch_attn_t)
}

cudaError_t launch_kv8_weights(int dt, const void* q, const int32_t* last, int n_q, const cb_kv8_cache& c, int H,
                               int Hkv, int hd, float* weights, void* ws, cudaStream_t s) {
  g_used_kv8_attn = true;
  const Kv8Attn p = make_params(q, last, n_q, c, H, Hkv, hd, nullptr, weights, ws);
  CB_KV8_DISPATCH(launch_weights_t)
}

}  // namespace cb
