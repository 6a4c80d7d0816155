// The 8-bit KV cache with one scale per block of rows and KV head: append, read back, and
// eviction by accumulated attention weight.  (Its attention: cb_kv8_attn.cu.)
//
//   value = code * scale,  scale = max(amax over the block's rows and the head's channels / 127, 1e-8)
//
// A scale per (block, head) instead of one per channel of a whole chunk (k_kv_quantize) lets
// rows be appended one at a time and lets attention apply it to a score or a probability: the
// codes themselves enter the matrix instructions, exactly.  The layout is head-major, so a
// head's block is one contiguous run of block * head_dim bytes.
#include <atomic>

#include "cb_kv8.cuh"

namespace cb {

static __device__ uint32_t g_err_kv8;
static std::atomic<bool> g_used_kv8{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_kv8() { return g_used_kv8 ? take_word(g_err_kv8) : 0u; }

namespace {

// rows [a, e) of sequence s that a call touches, from its start and count arrays
__device__ __forceinline__ bool kv8_rows(const int32_t* start, const int32_t* count, int n_rows, int64_t cap, int s,
                                         bool report, int64_t* a, int64_t* e) {
  const int64_t a0 = start[s];
  int64_t n = count ? count[s] : n_rows;
  bool bad = a0 < -1;
  if (a0 >= 0) {
    if (n < 0 || n > n_rows) {
      bad = true;
      n = n < 0 ? 0 : n_rows;
    }
    if (a0 + n > cap) bad = true;
  }
  if (bad && report) atomicOr(&g_err_kv8, ERRBIT_INDEX);
  if (a0 < 0) return false;
  *a = a0;
  *e = a0 + n < cap ? a0 + n : cap;
  return *a < *e;
}

// 16 consecutive elements as they were loaded, their largest magnitude as fp32 bits (above
// 0x7f7fffff if one is not finite), and their values (not finite: 0)
template <typename T>
struct Chunk;
template <>
struct Chunk<bf16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const bf16* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m) & 0x7fff7fffu;
    return max(u << 16, u & 0xffff0000u);
  }
  __device__ __forceinline__ void values(uint64_t* f) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = tc::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <>
struct Chunk<float> {
  uint4 w[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max(max(max(m, w[i].x & 0x7fffffffu), max(w[i].y & 0x7fffffffu, w[i].z & 0x7fffffffu)), w[i].w & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void values(uint64_t* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = tc::f2_pack(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
      f[2 * i + 1] = tc::f2_pack(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
    }
  }
};
// not finite: 0
__device__ __forceinline__ void zero_bad(uint64_t* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = tc::f2_unpack(f[i]);
    f[i] = tc::f2_pack(isfinite(v.x) ? v.x : 0.f, isfinite(v.y) ? v.y : 0.f);
  }
}

// One CTA per (touched block, K or V, head, sequence); a thread owns NCH chunks of 16 channels,
// held in registers between the maximum and the coding, so every new element is read once and
// every code written once.  Bound by HBM for a prompt: 4 x 16001 rows of 8 heads of 128 (262 MB
// of bf16 in, 131 MB of codes out) take about 65 us, 6 TB/s, in a replayed graph (two chunks per
// thread and 64-bit conversions where a tie shows: 110 us; conversions everywhere: 121 us); of fp32
// 107 us, 6.1 TB/s.  By latency for a token: one row of 4 sequences of 32 heads 4.1 us.
template <typename T, int NCH>
__global__ void __launch_bounds__(512, sizeof(T) == 2 ? 2 : 1) k_kv8_append(const T* __restrict__ k, const T* __restrict__ v, int n_rows,
                                                     const int32_t* __restrict__ start,
                                                     const int32_t* __restrict__ count, const cb_kv8_cache c, int lg,
                                                     int Hkv, int hd, uint32_t row_magic) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t sh[32];
  const int s = blockIdx.z, h = blockIdx.y, t = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  int64_t a, e;
  if (!kv8_rows(start, count, n_rows, c.capacity, s, blockIdx.x == 0 && h == 0 && threadIdx.x == 0, &a, &e)) return;
  const int64_t b = (a >> lg) + t, r0 = b << lg;
  if (r0 >= e) return;
  const int block = 1 << lg;
  const int lo = a > r0 ? (int)(a - r0) : 0;                       // rows [0, lo) of the block are older
  const int hi = e - r0 < block ? (int)(e - r0) : block;           // rows [lo, hi) are new
  const int64_t head = (int64_t)s * Hkv + h;
  int8_t* codes = (is_v ? c.v_codes : c.k_codes) + (head * c.capacity + r0) * hd;
  float* scale = (is_v ? c.v_scale : c.k_scale) + head * (c.capacity >> lg) + b;
  const float old = lo > 0 ? *scale : 0.f;
  const T* src = (is_v ? v : k) + (((int64_t)s * n_rows + (r0 - a)) * Hkv + h) * hd;
  // a thread's chunks lie whole rows apart
  const int row0 = threadIdx.x * row_magic >> 16, col = (threadIdx.x << 4) - row0 * hd, step = block / NCH;
  Chunk<T> x[NCH];
  uint32_t top = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int row = row0 + i * step;
    if (row >= lo && row < hi) x[i].load(src + (int64_t)row * Hkv * hd + col);
  }
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int row = row0 + i * step;
    if (row >= lo && row < hi) {
      uint32_t m = x[i].amax_bits();
      if (m >= 0x7f800000u) {
        bad = true;
        uint64_t f[8];
        x[i].values(f);
        zero_bad(f);
        m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 z = tc::f2_unpack(f[q]);
          m = max(max(m, __float_as_uint(z.x) & 0x7fffffffu), __float_as_uint(z.y) & 0x7fffffffu);
        }
      }
      top = max(top, m);
    }
  }
  if (bad) atomicOr(&g_err_kv8, ERRBIT_NONFINITE);
  const float amax = kv8_block_max(top, sh);
  const float sc = fmaxf(fmaxf(__fdiv_rn(amax, 127.0f), kKv8MinScale), old);
  const float inv = 1.0f / sc;
  const bool grow = sc > old;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int row = row0 + i * step;
    uint4* dst = reinterpret_cast<uint4*>(codes + row * hd + col);
    if (row >= lo && row < hi) {
      uint64_t f[8];
      x[i].values(f);
      if (bad) zero_bad(f);
      *dst = kv8_code16(f, inv, [&](float z, uint32_t q) { return kv8_code(z, sc, q); });
    } else if (row < lo && grow) {
      uint64_t g[8];
      kv8_unpack16(*dst, g);
      *dst = kv8_code16(g, old * inv, [&](float z, uint32_t q) { return kv8_recode(z, old, sc, q); });
    }
  }
  if (threadIdx.x == 0 && grow) *scale = sc;
}

// 8 consecutive values: one 32-byte store of floats where the buffer allows it
__device__ __forceinline__ void put8(bf16* p, const float* f, bool) { st8(p, f); }
__device__ __forceinline__ void put8(float* p, const float* f, bool al32) {
  if (al32)
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]),
                 "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  else
    st8(p, f);
}

// A thread turns 16 codes into 16 values, a few rows of them at once.  A CTA takes a run of
// rows of one head: the codes it reads are contiguous, each row it writes is a contiguous run
// of hd values.  Bound by HBM, mostly by what it writes: 655 MB in 97 us (fp32 out), 6.8 TB/s,
// with 32-byte stores; bf16 out, in 16-byte ones, 393 MB in 78 us, 5.1 TB/s.
constexpr int kReadUnroll = 4;
template <typename T>
__global__ void __launch_bounds__(256) k_kv8_read(const cb_kv8_cache c, int lg, const int32_t* __restrict__ start,
                                                  const int32_t* __restrict__ count, int n_rows, int Hkv, int hd,
                                                  T* __restrict__ k_out, T* __restrict__ v_out, bool al32) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.z, h = blockIdx.y >= (unsigned)Hkv ? blockIdx.y - Hkv : blockIdx.y;
  const bool is_v = k_out == nullptr || blockIdx.y >= (unsigned)Hkv;
  int64_t a, e;
  if (!kv8_rows(start, count, n_rows, c.capacity, s, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0, &a, &e))
    return;
  const int h16 = hd >> 4, per = 256 / h16;        // rows of one pass (hd 96 and the like leave threads idle)
  const int tr = threadIdx.x / h16, d = (threadIdx.x - tr * h16) << 4;
  const int64_t head = (int64_t)s * Hkv + h, row0 = (int64_t)blockIdx.x * per * kReadUnroll + tr;
  const int8_t* codes = (is_v ? c.v_codes : c.k_codes) + (head * c.capacity + a + row0) * hd + d;
  const float* scale = (is_v ? c.v_scale : c.k_scale) + head * (c.capacity >> lg);
  T* out = (is_v ? v_out : k_out) + (((int64_t)s * n_rows + row0) * Hkv + h) * hd + d;
  const int left = tr < per ? (int)(e - a - row0 < per * kReadUnroll ? e - a - row0 : per * kReadUnroll) : 0;   // rows from row0 on
  uint4 u[kReadUnroll];
  float sc[kReadUnroll];
#pragma unroll
  for (int i = 0; i < kReadUnroll; ++i)
    if (i * per < left) {
      u[i] = *reinterpret_cast<const uint4*>(codes + i * per * hd);
      sc[i] = scale[(a + row0 + i * per) >> lg];
    }
#pragma unroll
  for (int i = 0; i < kReadUnroll; ++i)
    if (i * per < left) {
      uint64_t g[8];
      float f[16];
      kv8_unpack16(u[i], g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 z = tc::f2_unpack(g[q]);
        f[2 * q] = __fmul_rn(z.x, sc[i]);
        f[2 * q + 1] = __fmul_rn(z.y, sc[i]);
      }
      T* o = out + (int64_t)i * per * Hkv * hd;
      put8(o, f, al32);
      put8(o + 8, f + 8, al32);
    }
}

// ---- eviction ---------------------------------------------------------------------------
// A weight is a sum of probabilities (>= 0), so its bit pattern orders it; NaN and negative
// values rank as 0.  One is added: 0 stands for a row that is not there.
__device__ __forceinline__ uint32_t weight_key(float w) { return (w > 0.f ? __float_as_uint(w) : 0u) + 1u; }

constexpr int kEvictBins = 2048;         // 11-bit digits: three passes over the 32 key bits

// One CTA per (head, sequence): radix select of the n_keep largest keys, where the first n_sink
// and the last n_recent rows have the largest key of all, ties to the lower row, then an
// ordered compaction.  A thread owns a run of consecutive rows, so it ranks its own keys by
// counting and one scan over the threads places them; their keys stay in registers over all
// passes (KPT of them: 4, 16 or 32 by the capacity; 8 heads of 16384 rows take 13 us with 16,
// 34 us read again in each pass, 32 heads of 32768 rows 29 and 77 us).  With KPT = 0 (more rows
// than 32 per thread) each pass reads the weights again.  Up to 1024 rows 256 threads do
// (eviction and read-back of 512 rows of 32 heads 10.4 us, 12.2 with 1024 threads, of 208 rows of 8 x 40
// heads 14.6 and 17.3; of 4096 rows of 32 heads 28.7 with 1024 threads, 31.2 with 256).
template <int NT, int KPT>
__global__ void __launch_bounds__(NT) k_kv8_select(const float* __restrict__ weights,
                                                              const int32_t* __restrict__ len, int64_t cap, int n_keep,
                                                              int n_sink, int n_recent, int64_t dcap,
                                                              int32_t* __restrict__ dst_len,
                                                              float* __restrict__ dst_weights,
                                                              int32_t* __restrict__ kept) {
  constexpr int BPT = kEvictBins / NT;           // bins of a thread
  __shared__ int hist[3][kEvictBins];
  __shared__ int s_sum[32], s_eq[32];
  __shared__ int s_digit, s_left;
  const int h = blockIdx.x, Hkv = gridDim.x, s = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < 3 * kEvictBins; i += NT) hist[0][i] = 0;
  pdl_wait();
  pdl_trigger();
  const int64_t head = (int64_t)s * Hkv + h;
  int64_t n = len[s];
  if (n < 0 || n > cap) {
    if (tid == 0 && h == 0) atomicOr(&g_err_kv8, ERRBIT_INDEX);
    n = n < 0 ? 0 : cap;
  }
  const float* w = weights + head * cap;
  int32_t* out = kept + head * n_keep;
  float* dw = dst_weights ? dst_weights + head * dcap : nullptr;
  const int n_out = n < n_keep ? (int)n : n_keep;
  if (tid == 0 && h == 0) dst_len[s] = n_out;
  for (int64_t i = n_out + tid; i < n_keep; i += NT) out[i] = -1;
  if (dw)
    for (int64_t i = n_out + tid; i < dcap; i += NT) dw[i] = 0.f;
  bool bad = false;
  auto look = [&](float v) { bad = bad || !(v >= 0.f) || isinf(v); };
  if (n <= n_keep) {
    for (int i = tid; i < (int)n; i += NT) {
      const float v = w[i];
      look(v);
      out[i] = i;
      if (dw) dw[i] = v;
    }
    if (bad) atomicOr(&g_err_kv8, ERRBIT_NONFINITE);
    return;
  }
  const int hi = (int)n - n_recent;
  auto key_of = [&](int i, float v) -> uint32_t {
    return i >= (int)n ? 0u : i < n_sink || i >= hi ? ~0u : weight_key(v);
  };
  // this thread's rows: whole float4's, within the capacity (a multiple of 16)
  const int run = KPT > 0 ? KPT : ((int)((n + NT - 1) / NT) + 3) & ~3, i0 = tid * run;
  uint32_t key[KPT > 0 ? KPT : 1];
  auto load4 = [&](int i) -> float4 {
    return i < (int)n ? *reinterpret_cast<const float4*>(w + i) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto look4 = [&](int i, float4 v) {
    look(v.x);
    if (i + 1 < (int)n) look(v.y);
    if (i + 2 < (int)n) look(v.z);
    if (i + 3 < (int)n) look(v.w);
  };
  auto each = [&](auto&& f) {                    // f(row, its key); rows past the last have key 0
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j) f(i0 + j, key[j]);
    } else {
      for (int i = i0; i < i0 + run && i < (int)n; i += 4) {
        const float4 v = load4(i);
        f(i, key_of(i, v.x));
        f(i + 1, key_of(i + 1, v.y));
        f(i + 2, key_of(i + 2, v.z));
        f(i + 3, key_of(i + 3, v.w));
      }
    }
  };
  if constexpr (KPT > 0) {
    float4 v[KPT / 4];
#pragma unroll
    for (int j = 0; j < KPT / 4; ++j) v[j] = load4(i0 + 4 * j);
#pragma unroll
    for (int j = 0; j < KPT / 4; ++j) {
      const int i = i0 + 4 * j;
      look4(i, v[j]);
      key[4 * j] = key_of(i, v[j].x);
      key[4 * j + 1] = key_of(i + 1, v[j].y);
      key[4 * j + 2] = key_of(i + 2, v[j].z);
      key[4 * j + 3] = key_of(i + 3, v[j].w);
    }
  } else {
    for (int i = i0; i < i0 + run && i < (int)n; i += 4) look4(i, load4(i));
  }
  if (bad) atomicOr(&g_err_kv8, ERRBIT_NONFINITE);
  __syncthreads();
  uint32_t prefix = 0, mask = 0;
  int left = n_keep;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t dmask = pass == 2 ? 1023u : 2047u;
    int* hp = hist[pass];
    each([&](int, uint32_t x) {
      if (x != 0u && (x & mask) == prefix) atomicAdd(&hp[(x >> shift) & dmask], 1);
    });
    __syncthreads();
    // thread t owns the BPT bins below 2048 - BPT t: inclusive scan from the top
    const int top = kEvictBins - 1 - BPT * tid;
    int c[BPT], own = 0;
#pragma unroll
    for (int i = 0; i < BPT; i += 2) {
      const int2 v = *reinterpret_cast<const int2*>(&hp[top - 1 - i]);
      c[i] = v.y;
      c[i + 1] = v.x;
      own += v.x + v.y;
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    incl += __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
    int excl = incl - own;
    if (excl < left && incl >= left) {     // exactly one thread
      int i = 0;
#pragma unroll
      for (int q = 0; q < BPT - 1; ++q)
        if (i == q && excl + c[q] < left) {
          excl += c[q];
          ++i;
        }
      s_digit = top - i;
      s_left = left - excl;
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    mask |= dmask << shift;
    left = s_left;
  }
  // every key above the threshold (fewer than n_keep) and the first `left` keys equal to it: a
  // thread's first place is the number of both before its rows
  int gt = 0, eq = 0;
  each([&](int, uint32_t x) {
    gt += x > prefix;
    eq += x == prefix;
  });
  int gi = gt, ei = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, gi, o), b = __shfl_up_sync(0xffffffffu, ei, o);
    if (lane >= o) {
      gi += a;
      ei += b;
    }
  }
  if (lane == 31) {
    s_sum[warp] = gi;
    s_eq[warp] = ei;
  }
  __syncthreads();
  int g = gi - gt + __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
  int q = ei - eq + __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  if constexpr (KPT > 0) {
    // kept rows as bits; then the warp walks its rows 32 at a time, so that the writes are in order
    const int at = g + min(q, left);
    uint32_t keep = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const bool same = key[j] == prefix;
      if (key[j] > prefix || (same && q < left)) keep |= 1u << j;
      q += same;
    }
    const int bit = lane % KPT;
#pragma unroll 4
    for (int j = 0; j < KPT; ++j) {
      const int from = j * (32 / KPT) + lane / KPT;
      const uint32_t m = __shfl_sync(0xffffffffu, keep, from);
      const int pos = __shfl_sync(0xffffffffu, at, from) + __popc(m & ((1u << bit) - 1u));
      if (m >> bit & 1u) {
        const int row = warp * 32 * KPT + j * 32 + lane;
        out[pos] = row;
        if (dw) dw[pos] = w[row];
      }
    }
  } else {
    each([&](int i, uint32_t x) {
      if (x > prefix || (x == prefix && q < left)) {
        const int pos = g + min(q, left);
        out[pos] = i;
        if (dw) dw[pos] = w[i];
      }
      g += x > prefix;
      q += x == prefix;
    });
  }
}

// the largest magnitude of 16 codes: bytes c + 128 as halves of words, their largest and smallest
__device__ __forceinline__ int max_code(const uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t hi = 0x00800080u, lo = 0x00800080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u, a = u & 0x00ff00ffu, b = __byte_perm(u, 0, 0x4341);
    hi = __vimax3_u16x2(hi, a, b);
    lo = __vimin3_u16x2(lo, a, b);
  }
  return max(max((int)(hi & 0xffffu), (int)(hi >> 16)) - 128, 128 - min((int)(lo & 0xffffu), (int)(lo >> 16)));
}

// One CTA per (destination block, K or V, head, sequence): gathers the block's kept rows,
// takes their largest value, codes them afresh.  Rows past the last kept one (kept[] < 0 there)
// are left alone.  A value is fl(code * its scale); its quotient by the new scale is coded from
// the code times the scales' ratio (kv8_code16's three roundings).  A CTA is a chain of three
// latencies (index, codes, maximum), so what counts is how many are resident: 64 registers (of
// 105 with K and V in one CTA: 129 us instead of 92).  4100 of 16384 rows of 16 x 8 heads (268 MB
// moved) take 72 us after the selection, 3.7 TB/s; deciding ties costs 14 us of them.
template <int NCH>
__global__ void __launch_bounds__(512, 2) k_kv8_move(const cb_kv8_cache c, const cb_kv8_cache d, int lg, int Hkv, int hd,
                                                  uint32_t row_magic, int n_keep, const int32_t* __restrict__ kept) {
  __shared__ uint32_t sh[32];
  const int s = blockIdx.z, h = blockIdx.y, b = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const int r0 = b << lg;
  const int64_t head = (int64_t)s * Hkv + h;
  const int8_t* codes = (is_v ? c.v_codes : c.k_codes) + head * c.capacity * hd;
  const float* scale = (is_v ? c.v_scale : c.k_scale) + head * (c.capacity >> lg);
  int8_t* out = (is_v ? d.v_codes : d.k_codes) + (head * d.capacity + r0) * hd;
  const int32_t* kr = kept + head * n_keep + r0;
  const int row0 = threadIdx.x * row_magic >> 16, col = (threadIdx.x << 4) - row0 * hd, step = (1 << lg) / NCH;
  pdl_wait();
  pdl_trigger();
  int r[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) r[i] = row0 + i * step < n_keep - r0 ? kr[row0 + i * step] : -1;
  if (kr[0] < 0) return;
  uint4 x[NCH];
  float xs[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if (r[i] >= 0) {
      xs[i] = scale[r[i] >> lg];
      x[i] = *reinterpret_cast<const uint4*>(codes + (int64_t)r[i] * hd + col);
    }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if (r[i] >= 0)       // the largest |code| times the scale is the largest |value|: products round monotonically
      top = max(top, __float_as_uint(__fmul_rn((float)max_code(x[i]), xs[i])) & 0x7fffffffu);
  const float amax = kv8_block_max(top, sh);
  const float sc = fmaxf(__fdiv_rn(amax, 127.0f), kKv8MinScale);
  const float inv = 1.0f / sc;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if (r[i] >= 0) {
      uint64_t f[8];
      kv8_unpack16(x[i], f);
      *reinterpret_cast<uint4*>(out + (row0 + i * step) * hd + col) =
          kv8_code16(f, xs[i] * inv, [&](float z, uint32_t q) { return kv8_code(__fmul_rn(z, xs[i]), sc, q); });
    }
  if (threadIdx.x == 0) (is_v ? d.v_scale : d.k_scale)[head * (d.capacity >> lg) + b] = sc;
}

// 16-channel chunks of a block (a multiple of 32, 32..2048) per thread, in whole warps and whole
// rows apart.  Four of them from 512 on for append, from 256 on for the move, whose loads wait for
// an index (blocks of 32 rows, hd 128: one token's append 4.1 us with two, 4.3 with four; halving
// a 4096-row cache 31.4 us with two, 29.3 with four).
int chunks_per_thread(int chunks, int four) {
  if (chunks >= four && chunks % 128 == 0) return 4;
  return chunks > 128 && chunks % 64 == 0 ? 2 : 1;
}
// t / (hd / 16) of a thread index t < 512 as t * magic >> 16
uint32_t row_magic(int hd) { return (65536 + hd / 16 - 1) / (hd / 16); }

int log2_of(int block) { return 31 - __builtin_clz((unsigned)block); }

}  // namespace

cudaError_t launch_kv8_append(int dt, const void* k, const void* v, int n_rows, const int32_t* start,
                              const int32_t* count, const cb_kv8_cache& c, int Hkv, int hd, cudaStream_t s) {
  g_used_kv8 = true;
  const int chunks = c.block * hd / 16, nch = chunks_per_thread(chunks, 512);
  // a run of n_rows rows touches at most this many blocks, wherever it starts
  const unsigned nb = (unsigned)(((int64_t)n_rows + 2 * c.block - 2) / c.block);
  const dim3 grid(2 * nb, Hkv, c.n_seq), blk(chunks / nch);
  const int lg = log2_of(c.block);
#define CB_APPEND(T, N)                                                                                      \
  return launch_k(k_kv8_append<T, N>, grid, blk, 0, s, static_cast<const T*>(k), static_cast<const T*>(v), n_rows, \
                  start, count, c, lg, Hkv, hd, row_magic(hd))
  if (dt == DT_BF16) {
    if (nch == 4) CB_APPEND(bf16, 4);
    if (nch == 2) CB_APPEND(bf16, 2);
    CB_APPEND(bf16, 1);
  }
  if (nch == 4) CB_APPEND(float, 4);
  if (nch == 2) CB_APPEND(float, 2);
  CB_APPEND(float, 1);
#undef CB_APPEND
}

cudaError_t launch_kv8_read(int dt, const cb_kv8_cache& c, const int32_t* start, const int32_t* count, int n_rows,
                            int Hkv, int hd, void* k_out, void* v_out, cudaStream_t s) {
  g_used_kv8 = true;
  const int per = 256 / (hd / 16) * kReadUnroll;
  const bool al32 = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  const dim3 grid((unsigned)(((int64_t)n_rows + per - 1) / per), k_out && v_out ? 2 * Hkv : Hkv, c.n_seq);
  const int lg = log2_of(c.block);
  if (dt == DT_BF16)
    return launch_k(k_kv8_read<bf16>, grid, dim3(256), 0, s, c, lg, start, count, n_rows, Hkv, hd,
                    static_cast<bf16*>(k_out), static_cast<bf16*>(v_out), al32);
  return launch_k(k_kv8_read<float>, grid, dim3(256), 0, s, c, lg, start, count, n_rows, Hkv, hd,
                  static_cast<float*>(k_out), static_cast<float*>(v_out), al32);
}

cudaError_t launch_kv8_select(const cb_kv8_cache& c, const int32_t* len, const float* weights, int n_keep, int n_sink,
                              int n_recent, int64_t dcap, int32_t* dst_len, float* dst_weights, int32_t* kept, int Hkv,
                              cudaStream_t s) {
  g_used_kv8 = true;
  const dim3 grid(Hkv, c.n_seq);
#define CB_SELECT(NT, KPT)                                                                                          \
  return launch_k(k_kv8_select<NT, KPT>, grid, dim3(NT), 0, s, weights, len, c.capacity, n_keep, n_sink, n_recent, dcap, \
                  dst_len, dst_weights, kept)
  if (c.capacity <= 4 * 256) CB_SELECT(256, 4);
  if (c.capacity <= 4 * 1024) CB_SELECT(1024, 4);
  if (c.capacity <= 16 * 1024) CB_SELECT(1024, 16);
  if (c.capacity <= 32 * 1024) CB_SELECT(1024, 32);
  CB_SELECT(1024, 0);
#undef CB_SELECT
}

cudaError_t launch_kv8_move(const cb_kv8_cache& c, const cb_kv8_cache& d, int n_keep, const int32_t* kept, int Hkv,
                            int hd, cudaStream_t s) {
  g_used_kv8 = true;
  const int chunks = c.block * hd / 16, nch = chunks_per_thread(chunks, 256);
  const dim3 grid(2 * ((n_keep + c.block - 1) / c.block), Hkv, c.n_seq), blk(chunks / nch);
  const int lg = log2_of(c.block);
#define CB_MOVE(N) return launch_k(k_kv8_move<N>, grid, blk, 0, s, c, d, lg, Hkv, hd, row_magic(hd), n_keep, kept)
  if (nch == 4) CB_MOVE(4);
  if (nch == 2) CB_MOVE(2);
  CB_MOVE(1);
#undef CB_MOVE
}

}  // namespace cb
