// The 8-bit KV cache with one scale per block of rows and KV head: append, read back, and
// eviction by accumulated attention weight.  (Its attention: cb_kv8_attn.cu.)
//
//   value = code * scale,  scale = max(amax over the block's rows and the head's channels / 127, 1e-8)
//
// A scale per (block, head) instead of one per channel of a whole chunk (k_kv_quantize) lets
// rows be appended one at a time and lets attention apply it to a score or a probability: the
// codes themselves enter the matrix instructions, exactly.  The layout is head-major, so a
// head's block is one contiguous run of block * head_dim bytes.
#include <mutex>

#include "cb_kv8.cuh"

namespace cb {

static __device__ uint32_t g_err_kv8;

uint32_t take_error_kv8() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv8, sizeof(v)) != cudaSuccess) return ERRBIT_INDEX;
  cudaMemcpyToSymbol(g_err_kv8, &z, sizeof(z));
  return v;
}

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
  __device__ __forceinline__ void values(float* f) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
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
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = __uint_as_float(w[i].x);
      f[4 * i + 1] = __uint_as_float(w[i].y);
      f[4 * i + 2] = __uint_as_float(w[i].z);
      f[4 * i + 3] = __uint_as_float(w[i].w);
    }
  }
};
// not finite: 0
__device__ __forceinline__ void zero_bad(float* f) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (!isfinite(f[i])) f[i] = 0.f;
}

// One CTA per (touched block, K or V, head, sequence); a thread owns NCH chunks of 16 channels
// of one row, held in registers between the maximum and the coding, so every new element is
// read once.
template <typename T, int NCH>
__global__ void __launch_bounds__(1024) k_kv8_append(const T* __restrict__ k, const T* __restrict__ v, int n_rows,
                                                     const int32_t* __restrict__ start,
                                                     const int32_t* __restrict__ count, const cb_kv8_cache c, int lg,
                                                     int Hkv, int hd) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sh[32];
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
  const int per_row = hd >> 4;
  const T* src = (is_v ? v : k) + (((int64_t)s * n_rows + (r0 - a)) * Hkv + h) * hd;
  // a thread's chunks lie whole rows apart
  const int row0 = threadIdx.x / per_row, col = (threadIdx.x - row0 * per_row) << 4, step = block / NCH;
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
        float f[16];
        x[i].values(f);
        zero_bad(f);
        float a = 0.f;
#pragma unroll
        for (int q = 0; q < 16; ++q) a = fmaxf(a, fabsf(f[q]));
        m = __float_as_uint(a);
      }
      top = max(top, m);
    }
  }
  if (bad) atomicOr(&g_err_kv8, ERRBIT_NONFINITE);
  const float amax = kv8_block_max(__uint_as_float(top), sh);
  const float sc = fmaxf(fmaxf(__fdiv_rn(amax, 127.0f), kKv8MinScale), old);
  const float inv = 1.0f / sc;
  const bool grow = sc > old;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int row = row0 + i * step;
    uint4* dst = reinterpret_cast<uint4*>(codes + row * hd + col);
    if (row >= lo && row < hi) {
      float f[16];
      x[i].values(f);
      if (bad) zero_bad(f);
      *dst = kv8_code16(f, sc, inv);
    } else if (row < lo && grow) {
      float g[16];
      uint32_t q[16];
      kv8_unpack16(*dst, g);
#pragma unroll
      for (int c = 0; c < 16; ++c) q[c] = (uint32_t)(int)kv8_recode(g[c], old, sc, inv);
      *dst = make_uint4(kv8_pack4(q[0], q[1], q[2], q[3]), kv8_pack4(q[4], q[5], q[6], q[7]),
                        kv8_pack4(q[8], q[9], q[10], q[11]), kv8_pack4(q[12], q[13], q[14], q[15]));
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
// of hd values.
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
      float f[16];
      kv8_unpack16(u[i], f);
#pragma unroll
      for (int q = 0; q < 16; ++q) f[q] = __fmul_rn(f[q], sc[i]);
      T* o = out + (int64_t)i * per * Hkv * hd;
      put8(o, f, al32);
      put8(o + 8, f + 8, al32);
    }
}

// ---- eviction ---------------------------------------------------------------------------
// A weight is a sum of probabilities (>= 0), so its bit pattern orders it; NaN and negative
// values rank as 0.
__device__ __forceinline__ uint32_t weight_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

constexpr int kEvictThreads = 1024;
constexpr int kEvictSmemKeys = 49152;    // keys staged in shared memory up to this many (192 KB)
constexpr int kEvictBins = 2048;         // 11-bit digits: three passes over the 32 key bits

// One CTA per (head, sequence): radix select of the k heaviest rows of [lo, hi), ties to the
// lower row, then an ordered compaction: warp w owns a contiguous run of rows and ranks them
// by ballots, so no lane strides through shared memory.
template <bool SMEM>
__global__ void __launch_bounds__(kEvictThreads) k_kv8_select(const float* __restrict__ weights,
                                                              const int32_t* __restrict__ len, int64_t cap, int n_keep,
                                                              int n_sink, int n_recent, int64_t dcap,
                                                              int32_t* __restrict__ dst_len,
                                                              float* __restrict__ dst_weights,
                                                              int32_t* __restrict__ kept) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t skey[];
  __shared__ int hist[kEvictBins];
  __shared__ int s_gt[32], s_eq[32];
  __shared__ int s_digit, s_left;
  const int h = blockIdx.x, Hkv = gridDim.x, s = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
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
  for (int64_t i = n_out + tid; i < n_keep; i += kEvictThreads) out[i] = -1;
  if (dw)
    for (int64_t i = n_out + tid; i < dcap; i += kEvictThreads) dw[i] = 0.f;
  auto emit = [&](int pos, int row) {
    out[pos] = row;
    if (dw) dw[pos] = w[row];
  };
  bool bad = false;
  if (n <= n_keep) {
    for (int i = tid; i < (int)n; i += kEvictThreads) {
      if (!(w[i] >= 0.f) || isinf(w[i])) bad = true;
      emit(i, i);
    }
    if (bad) atomicOr(&g_err_kv8, ERRBIT_NONFINITE);
    return;
  }
  const int lo = n_sink, hi = (int)n - n_recent, m = hi - lo;    // candidates; m > k because n > n_keep
  const int k = n_keep - n_sink - n_recent;
  for (int i = tid; i < n_sink; i += kEvictThreads) emit(i, i);
  for (int i = tid; i < n_recent; i += kEvictThreads) emit(n_keep - n_recent + i, hi + i);
  for (int i = tid; i < (int)n; i += kEvictThreads) {
    const float v = w[i];
    if (!(v >= 0.f) || isinf(v)) bad = true;
    if (SMEM && i >= lo && i < hi) skey[i - lo] = weight_key(v);
  }
  if (bad) atomicOr(&g_err_kv8, ERRBIT_NONFINITE);
  if (k == 0) return;
  auto key_at = [&](int i) -> uint32_t { return SMEM ? skey[i] : weight_key(w[lo + i]); };
  uint32_t prefix = 0, mask = 0;
  int left = k;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t dmask = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kEvictThreads) {
      const uint32_t key = key_at(i);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & dmask], 1);
    }
    __syncthreads();
    // thread t owns bins 2047 - 2t and 2046 - 2t: inclusive scan from the top
    const int c0 = hist[kEvictBins - 1 - 2 * tid], c1 = hist[kEvictBins - 2 - 2 * tid];
    int incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_gt[warp] = incl;
    __syncthreads();
    int base = 0;
    for (int i = 0; i < warp; ++i) base += s_gt[i];
    incl += base;
    const int excl = incl - c0 - c1;
    if (excl < left && incl >= left) {     // exactly one thread
      const bool second = excl + c0 < left;
      s_digit = kEvictBins - 1 - 2 * tid - (second ? 1 : 0);
      s_left = left - excl - (second ? c0 : 0);
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    mask |= dmask << shift;
    left = s_left;
    __syncthreads();
  }
  // every key above the threshold, and the first `left` keys equal to it
  const int seg = ((m + 31) / 32 + 31) & ~31;    // rows per warp, a multiple of 32
  const int i0 = warp * seg, i1 = min(m, i0 + seg);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t key = in ? key_at(i + lane) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, in && key > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;
  for (int i = 0; i < warp; ++i) {
    gt0 += s_gt[i];
    eq0 += s_eq[i];
  }
  const unsigned below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t key = in ? key_at(i + lane) : 0u;
    const unsigned bg = __ballot_sync(0xffffffffu, in && key > prefix);
    const unsigned be = __ballot_sync(0xffffffffu, in && key == prefix);
    const int g = gt0 + __popc(bg & below), q = eq0 + __popc(be & below);    // before this row
    if (((bg >> lane) & 1) || (((be >> lane) & 1) && q < left)) emit(n_sink + g + min(q, left), lo + i + lane);
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
}

// One CTA per (destination block, K or V, head, sequence): gathers the block's kept rows,
// takes their largest value, codes them afresh.  Rows past the last kept one are left alone.
template <int NCH>
__global__ void __launch_bounds__(1024) k_kv8_move(const cb_kv8_cache c, const cb_kv8_cache d, int lg, int Hkv, int hd,
                                                   const int32_t* __restrict__ dst_len, int n_keep,
                                                   const int32_t* __restrict__ kept) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sh[32];
  const int s = blockIdx.z, h = blockIdx.y, b = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const int r0 = b << lg, n = dst_len[s];
  if (r0 >= n) return;
  const int rows = min(1 << lg, n - r0);
  const int64_t head = (int64_t)s * Hkv + h;
  const int8_t* codes = (is_v ? c.v_codes : c.k_codes) + head * c.capacity * hd;
  const float* scale = (is_v ? c.v_scale : c.k_scale) + head * (c.capacity >> lg);
  int8_t* out = (is_v ? d.v_codes : d.k_codes) + (head * d.capacity + r0) * hd;
  const int32_t* kr = kept + head * n_keep + r0;
  const int per_row = hd >> 4;
  const int row0 = threadIdx.x / per_row, col = (threadIdx.x - row0 * per_row) << 4, step = (1 << lg) / NCH;
  uint4 x[NCH];
  float f[NCH][16], xs[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int row = row0 + i * step;
    if (row < rows) {
      const int64_t r = kr[row];
      xs[i] = scale[r >> lg];
      x[i] = *reinterpret_cast<const uint4*>(codes + r * hd + col);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if (row0 + i * step < rows) {
      // the largest |code| times the scale is the largest |value|: products round monotonically
      float m = 0.f;
      kv8_unpack16(x[i], f[i]);
#pragma unroll
      for (int q = 0; q < 16; ++q) m = fmaxf(m, fabsf(f[i][q]));
      amax = fmaxf(amax, __fmul_rn(m, xs[i]));
    }
  amax = kv8_block_max(amax, sh);
  const float sc = fmaxf(__fdiv_rn(amax, 127.0f), kKv8MinScale);
  const float inv = 1.0f / sc;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int row = row0 + i * step;
    if (row < rows) {
#pragma unroll
      for (int q = 0; q < 16; ++q) f[i][q] = __fmul_rn(f[i][q], xs[i]);
      *reinterpret_cast<uint4*>(out + row * hd + col) = kv8_code16(f[i], sc, inv);
    }
  }
  if (threadIdx.x == 0) (is_v ? d.v_scale : d.k_scale)[head * (d.capacity >> lg) + b] = sc;
}

// select's shared-memory limit set, per device
std::mutex g_kv8_mem_mu;
bool g_select_attr[64];

// 16-channel chunks of a block (a multiple of 32, 32..2048) per thread, in whole warps
int chunks_per_thread(int chunks) { return chunks > 128 && chunks % 64 == 0 ? 2 : 1; }

int log2_of(int block) { return 31 - __builtin_clz((unsigned)block); }

}  // namespace

void reset_kv8_caches() {
  std::lock_guard<std::mutex> g(g_kv8_mem_mu);
  for (int i = 0; i < 64; ++i) g_select_attr[i] = false;
}

cudaError_t launch_kv8_append(int dt, const void* k, const void* v, int n_rows, const int32_t* start,
                              const int32_t* count, const cb_kv8_cache& c, int Hkv, int hd, cudaStream_t s) {
  const int chunks = c.block * hd / 16, nch = chunks_per_thread(chunks);
  // a run of n_rows rows touches at most this many blocks, wherever it starts
  const unsigned nb = (unsigned)(((int64_t)n_rows + 2 * c.block - 2) / c.block);
  const dim3 grid(2 * nb, Hkv, c.n_seq), blk(chunks / nch);
  const int lg = log2_of(c.block);
#define CB_APPEND(T, N)                                                                                      \
  return launch_k(k_kv8_append<T, N>, grid, blk, 0, s, static_cast<const T*>(k), static_cast<const T*>(v), n_rows, \
                  start, count, c, lg, Hkv, hd)
  if (dt == DT_BF16) {
    if (nch == 2) CB_APPEND(bf16, 2);
    CB_APPEND(bf16, 1);
  }
  if (nch == 2) CB_APPEND(float, 2);
  CB_APPEND(float, 1);
#undef CB_APPEND
}

cudaError_t launch_kv8_read(int dt, const cb_kv8_cache& c, const int32_t* start, const int32_t* count, int n_rows,
                            int Hkv, int hd, void* k_out, void* v_out, cudaStream_t s) {
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
  const dim3 grid(Hkv, c.n_seq);
  if (c.capacity > kEvictSmemKeys)
    return launch_k(k_kv8_select<false>, grid, dim3(kEvictThreads), 0, s, weights, len, c.capacity, n_keep, n_sink,
                    n_recent, dcap, dst_len, dst_weights, kept);
  const size_t smem = (size_t)c.capacity * 4;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> g(g_kv8_mem_mu);
    if (dev < 0 || dev >= 64 || !g_select_attr[dev]) {
      e = cudaFuncSetAttribute(k_kv8_select<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictSmemKeys * 4);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) g_select_attr[dev] = true;
    }
  }
  return launch_k(k_kv8_select<true>, grid, dim3(kEvictThreads), smem, s, weights, len, c.capacity, n_keep, n_sink,
                  n_recent, dcap, dst_len, dst_weights, kept);
}

cudaError_t launch_kv8_move(const cb_kv8_cache& c, const cb_kv8_cache& d, const int32_t* dst_len, int n_keep,
                            const int32_t* kept, int Hkv, int hd, cudaStream_t s) {
  const int chunks = c.block * hd / 16, nch = chunks_per_thread(chunks);
  const dim3 grid(2 * ((n_keep + c.block - 1) / c.block), Hkv, c.n_seq), blk(chunks / nch);
  const int lg = log2_of(c.block);
  if (nch == 2) return launch_k(k_kv8_move<2>, grid, blk, 0, s, c, d, lg, Hkv, hd, dst_len, n_keep, kept);
  return launch_k(k_kv8_move<1>, grid, blk, 0, s, c, d, lg, Hkv, hd, dst_len, n_keep, kept);
}

}  // namespace cb
