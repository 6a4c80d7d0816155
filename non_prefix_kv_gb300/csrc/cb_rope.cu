// Rotary positions in any of the usual forms: pairs (x[2i], x[2i + 1]) or (x[i], x[i + rot / 2]) of a
// head's first rot channels, with a table whose frequencies may be scaled for long contexts; query rows
// beside key and value rows, which may come from listed rows and go to listed rows (of a cache).
//
// y1 = x1 c - x2 s, y2 = x1 s + x2 c with c, s of the row's position from the table; a negative position
// or an inverse call negates s.  fp32 arithmetic, one rounding at the end.
//
// HBM-bound: every row is read once and written once, the table's row (4 rot bytes) comes from L2.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "../../include/cacheblend.h"
#include "cb_common.cuh"
#include "cb_internal.h"

namespace cb {

static __device__ uint32_t g_err_rope;
static std::atomic<bool> g_used_rope{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_rope() { return g_used_rope ? take_word(g_err_rope) : 0u; }

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

struct Thetas {
  double t[kMaxPairs];
};

// cos and sin of p theta_i, the angle formed in 64 bits, times the amplitude, rounded once
__global__ void __launch_bounds__(256) k_rope_table_scaled(float2* tab, int64_t n, int half, double amplitude,
                                                           const __grid_constant__ Thetas th) {
  pdl_wait();
  pdl_trigger();
  for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < n; t += (int64_t)gridDim.x * blockDim.x) {
    const int64_t p = t / half;
    double s, c;
    sincos((double)p * th.t[t - p * half], &s, &c);
    tab[t] = make_float2((float)(c * amplitude), (float)(s * amplitude));
  }
}

struct RopeRows {
  cb_rope_rows_io io;
  const int32_t* pos;
  const float2* tab;
  int n, H, Hkv, hd, rot, max_pos;
  int cols;                 // items of a rotated head: its pairs (in groups of V), then its other channels
  int inverse;
};

// V elements as they are in memory
template <typename T, int V>
struct Raw {
  uint4 q[sizeof(T) * V / 16];
  template <bool STREAM>
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * V / 16; ++i)
      q[i] = STREAM ? __ldcs(reinterpret_cast<const uint4*>(p) + i) : reinterpret_cast<const uint4*>(p)[i];
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * V / 16; ++i) {
      if (STREAM)
        __stcs(reinterpret_cast<uint4*>(p) + i, q[i]);
      else
        reinterpret_cast<uint4*>(p)[i] = q[i];
    }
  }
  __device__ __forceinline__ void get(float* x) const { ld8(reinterpret_cast<const T*>(q), x); }
  __device__ __forceinline__ void set(const float* x) { st8(reinterpret_cast<T*>(q), x); }
};
template <typename T>
struct Raw<T, 1> {
  T q;
  template <bool STREAM>
  __device__ __forceinline__ void load(const T* p) { q = *p; }
  template <bool STREAM>
  __device__ __forceinline__ void store(T* p) const { *p = q; }
  __device__ __forceinline__ void get(float* x) const { x[0] = to_f(q); }
  __device__ __forceinline__ void set(const float* x) { q = from_f<T>(x[0]); }
};

// An item of a rotated head is V pairs (V = 8: two 16-byte words of bf16) or V of the channels that stay;
// of a value head V channels.  A thread keeps its place in the head and walks the heads, so that it reads
// its part of the table's row once.  V = 1 serves what is not aligned to eight elements.
//
// A row's loads come before its stores: values first, then two heads at a time (one after the other, each with
// its own round trip, 16001 rows of 72 heads took 112 us and 3840 rows of 2 x 32, half of each rotated, 34; so
// 109 and 25).  Calls that move more than L2 holds do not leave their rows there (96 and 21; for a token's rows,
// which attention reads next, that would be the wrong way round: 2.2 us, 2.5 with it).  96 us are 6.1 TB/s.
template <typename T, int V, bool HALF, bool STREAM>
__global__ void __launch_bounds__(kThreads) k_rope_rows(const RopeRows p) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, half = p.rot / 2;
  const cb_rope_rows_io& io = p.io;
  const int heads = (io.q ? p.H : 0) + (io.k ? p.Hkv : 0);
  const int pairs = half / V, tid = threadIdx.x, threads = blockDim.x;
  const int64_t sr = io.src_row ? io.src_row[row] : row;
  const int64_t dr = io.kv_row ? io.kv_row[row] : row;
  const int pos = p.pos[row], ap = pos < 0 ? -pos : pos;
  const bool bad_pos = pos <= -p.max_pos || pos >= p.max_pos;
  const bool bad_row = io.k && (sr < 0 || sr >= io.n_src_rows || dr < -1 || dr >= io.n_out_rows);
  if ((bad_pos || bad_row) && blockIdx.y == 0 && tid == 0) atomicOr(&g_err_rope, ERRBIT_INDEX);
  if (bad_pos) return;
  const bool kv_on = io.k && !bad_row && dr >= 0;       // dr = -1: an idle row, nothing is stored
  // ---- values, on their way
  constexpr int NV = 2;
  Raw<T, V> val[NV];
  const int W = io.v && kv_on ? p.Hkv * p.hd : 0, v0 = (blockIdx.y * threads + tid) * V, vs = gridDim.y * threads * V;
  const T* vx = static_cast<const T*>(io.v) + sr * io.v_ld;
  T* vy = static_cast<T*>(io.v_out) + dr * io.kv_out_ld;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (v0 + j * vs < W) val[j].template load<STREAM>(vx + v0 + j * vs);
  // ---- rotated heads
  const int per = threads / p.cols, col = tid % p.cols;
  const float sg = (pos < 0) != (p.inverse != 0) ? -1.0f : 1.0f;
  const bool turn = col < pairs;
  float c[V], s[V];
  if (turn) {
    const float2* tb = p.tab + (int64_t)ap * half + col * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 cs = tb[i];
      c[i] = cs.x;
      s[i] = cs.y * sg;
    }
  }
  // the item's first channel, and the one of its pairs' other halves
  const int at = turn ? (HALF ? col * V : 2 * col * V) : p.rot + (col - pairs) * V;
  const int by = HALF ? half : V;
  const int first = io.q ? 0 : p.H, step = gridDim.y * per, last = kv_on ? heads : heads - (io.k ? p.Hkv : 0);
  auto from = [&](int h) -> const T* {
    return (h < p.H ? static_cast<const T*>(io.q) + (int64_t)row * io.q_ld + h * p.hd
                    : static_cast<const T*>(io.k) + sr * io.k_ld + (h - p.H) * p.hd) + at;
  };
  auto to = [&](int h) -> T* {
    return (h < p.H ? static_cast<T*>(io.q_out) + (int64_t)row * io.q_out_ld + h * p.hd
                    : static_cast<T*>(io.k_out) + dr * io.kv_out_ld + (h - p.H) * p.hd) + at;
  };
  auto rotate = [&](Raw<T, V>& x, Raw<T, V>& y) {
    float a[V], b[V];
    x.get(a);
    y.get(b);
    if constexpr (HALF || V == 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float u = a[j], w = b[j];
        a[j] = u * c[j] - w * s[j];
        b[j] = u * s[j] + w * c[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        float u = a[2 * j], w = a[2 * j + 1];
        a[2 * j] = u * c[j] - w * s[j];
        a[2 * j + 1] = u * s[j] + w * c[j];
        u = b[2 * j], w = b[2 * j + 1];
        b[2 * j] = u * c[V / 2 + j] - w * s[V / 2 + j];
        b[2 * j + 1] = u * s[V / 2 + j] + w * c[V / 2 + j];
      }
    }
    x.set(a);
    y.set(b);
  };
  for (int i = tid / p.cols < per ? blockIdx.y * per + tid / p.cols : last; i < last; i += 2 * step) {
    const bool two = i + step < last;
    Raw<T, V> a0, b0, a1, b1;
    a0.template load<STREAM>(from(first + i));
    if (turn) b0.template load<STREAM>(from(first + i) + by);
    if (two) {
      a1.template load<STREAM>(from(first + i + step));
      if (turn) b1.template load<STREAM>(from(first + i + step) + by);
    }
    if (turn) {
      rotate(a0, b0);
      b0.template store<STREAM>(to(first + i) + by);
    }
    a0.template store<STREAM>(to(first + i));
    if (two) {
      if (turn) {
        rotate(a1, b1);
        b1.template store<STREAM>(to(first + i + step) + by);
      }
      a1.template store<STREAM>(to(first + i + step));
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (v0 + j * vs < W) val[j].template store<STREAM>(vy + v0 + j * vs);
  for (int i = v0 + NV * vs; i < W; i += vs) {
    val[0].template load<STREAM>(vx + i);
    val[0].template store<STREAM>(vy + i);
  }
}

template <typename T, int V>
cudaError_t launch_v(RopeRows p, bool half, cudaStream_t s) {
  p.cols = p.rot / 2 / V + (p.hd - p.rot) / V;
  const int heads = (p.io.q ? p.H : 0) + (p.io.k ? p.Hkv : 0);
  // a thread for every item of a small row (1001 rows of 8 heads of 64: 6.8 us with 256 threads a row)
  const int threads = std::min(kThreads, std::max((heads * p.cols + 31) / 32, (p.cols + 31) / 32) * 32);
  const int rounds = (heads + threads / p.cols - 1) / (threads / p.cols);
  // few rows: a CTA for every round of the heads, so that the row's loads are all in flight at once
  const int split = p.n >= 1024 ? 1 : std::min(rounds, std::max(1, 1024 / p.n));
  const dim3 grid(p.n, split);
  const double moved = 2.0 * sizeof(T) * p.n * p.hd * (heads + (p.io.v ? p.Hkv : 0));
  if (V == 8 && moved > 100e6)
    return half ? launch_k(k_rope_rows<T, V, true, V == 8>, grid, dim3(threads), 0, s, p)
                : launch_k(k_rope_rows<T, V, false, V == 8>, grid, dim3(threads), 0, s, p);
  return half ? launch_k(k_rope_rows<T, V, true, false>, grid, dim3(threads), 0, s, p)
              : launch_k(k_rope_rows<T, V, false, false>, grid, dim3(threads), 0, s, p);
}

}  // namespace

cudaError_t launch_rope_table_scaled(float* tab, int max_pos, int rot, const double* theta, double amplitude,
                                     cudaStream_t s) {
  g_used_rope = true;
  Thetas th;
  for (int i = 0; i < rot / 2; ++i) th.t[i] = theta[i];
  const int64_t n = (int64_t)max_pos * (rot / 2);
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20);
  return launch_k(k_rope_table_scaled, dim3(grid), dim3(256), 0, s, reinterpret_cast<float2*>(tab), n, rot / 2, amplitude,
                  th);
}

// vec: every row starts on 16 bytes and the pairs come in groups of eight
cudaError_t launch_rope_rows(int dt, const cb_rope_rows_io& io, const int32_t* pos, int n, int H, int Hkv, int hd, int rot,
                             bool half, bool vec, const float* tab, int max_pos, bool inverse, cudaStream_t s) {
  g_used_rope = true;
  RopeRows p{io, pos, reinterpret_cast<const float2*>(tab), n, H, Hkv, hd, rot, max_pos, 0, inverse};
  if (dt == DT_BF16) return vec ? launch_v<bf16, 8>(p, half, s) : launch_v<bf16, 1>(p, half, s);
  return vec ? launch_v<float, 8>(p, half, s) : launch_v<float, 1>(p, half, s);
}

}  // namespace cb
