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

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float* x) {
  if constexpr (V == 8)
    ld8(p, x);
  else
    x[0] = to_f(p[0]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float* x) {
  if constexpr (V == 8)
    st8(p, x);
  else
    p[0] = from_f<T>(x[0]);
}

// An item of a rotated head is V pairs (V = 8: two 16-byte words of bf16) or V of the channels that stay;
// of a value head V channels.  A thread keeps its place in the head and walks the heads, so that it reads
// its part of the table's row once.  V = 1 serves what is not aligned to eight elements.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rope_rows(const RopeRows p) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, half = p.rot / 2;
  const cb_rope_rows_io& io = p.io;
  const int heads = (io.q ? p.H : 0) + (io.k ? p.Hkv : 0);
  const int pairs = half / V, tid = threadIdx.x;
  const int64_t sr = io.src_row ? io.src_row[row] : row;
  const int64_t dr = io.kv_row ? io.kv_row[row] : row;
  const int pos = p.pos[row], ap = pos < 0 ? -pos : pos;
  const bool bad_pos = pos <= -p.max_pos || pos >= p.max_pos;
  const bool bad_row = io.k && (sr < 0 || sr >= io.n_src_rows || dr < -1 || dr >= io.n_out_rows);
  if ((bad_pos || bad_row) && blockIdx.y == 0 && tid == 0) atomicOr(&g_err_rope, ERRBIT_INDEX);
  if (bad_pos) return;
  const bool kv_on = io.k && !bad_row && dr >= 0;       // dr = -1: an idle row, nothing is stored
  // ---- rotated heads
  const int per = kThreads / p.cols, col = tid % p.cols;
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
  const int first = io.q ? 0 : p.H;
  for (int i = blockIdx.y * per + tid / p.cols; tid / p.cols < per && i < heads; i += gridDim.y * per) {
    const int h = first + i;
    const bool q = h < p.H;
    if (!q && !kv_on) break;
    const T* x = (q ? static_cast<const T*>(io.q) + (int64_t)row * io.q_ld + h * p.hd
                    : static_cast<const T*>(io.k) + sr * io.k_ld + (h - p.H) * p.hd) + at;
    T* y = (q ? static_cast<T*>(io.q_out) + (int64_t)row * io.q_out_ld + h * p.hd
              : static_cast<T*>(io.k_out) + dr * io.kv_out_ld + (h - p.H) * p.hd) + at;
    if (turn) {
      float a[V], b[V];
      load<T, V>(x, a);
      load<T, V>(x + by, b);
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
      store<T, V>(y, a);
      store<T, V>(y + by, b);
    } else {
      float a[V];
      load<T, V>(x, a);
      store<T, V>(y, a);
    }
  }
  // ---- values
  if (!io.v || !kv_on) return;
  const T* x = static_cast<const T*>(io.v) + sr * io.v_ld;
  T* y = static_cast<T*>(io.v_out) + dr * io.kv_out_ld;
  const int W = p.Hkv * p.hd;
  for (int i = (blockIdx.y * kThreads + tid) * V; i < W; i += gridDim.y * kThreads * V) {
    float a[V];
    load<T, V>(x + i, a);
    store<T, V>(y + i, a);
  }
}

template <typename T, int V>
cudaError_t launch_v(RopeRows p, bool half, cudaStream_t s) {
  p.cols = p.rot / 2 / V + (p.hd - p.rot) / V;
  const int heads = (p.io.q ? p.H : 0) + (p.io.k ? p.Hkv : 0);
  const int rounds = (heads + kThreads / p.cols - 1) / (kThreads / p.cols);
  // few rows: a CTA for every round of the heads, so that the row's loads are all in flight at once
  const int split = p.n >= 1024 ? 1 : std::min(rounds, std::max(1, 1024 / p.n));
  const dim3 grid(p.n, split);
  return half ? launch_k(k_rope_rows<T, V, true>, grid, dim3(kThreads), 0, s, p)
              : launch_k(k_rope_rows<T, V, false>, grid, dim3(kThreads), 0, s, p);
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
