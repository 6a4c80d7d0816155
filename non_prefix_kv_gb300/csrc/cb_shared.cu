// Attention of a batch of sequences that share long prefixes, each with its own rows behind:
//
//   out = sum_i p_i v_i,  p = softmax_i(q . k_i / sqrt(hd)),  i over the prefix of the sequence's group and
//   its own rows 0..last
//
// The softmax is taken piece by piece: a piece (some keys of one kind, some rows) leaves its rows' largest
// exponent m (of 2), the sum l of 2^(z - m) and the weighted sum o of v; pieces join as
//   out = sum o 2^(m - M) / sum l 2^(m - M),  M = max m.
// So the prefix is one matrix product with every row of the group's batch, its keys and values read once
// per 16 (here) rows of one KV head, and each sequence's own rows are a small product of their own.
//
// This file: fp32 rows (exact arithmetic) and head sizes that the tensor-core kernels do not take.  4 rows of 8
// lanes share a warp, K and then V of 32 keys in shared memory: 6 x 3 queries of 4 heads of 64 over 1000 rows take
// 11.7 us, most of it two launches and the chain of loads of one piece; a call of many rows is bound by the fp32
// products, which read a key's value from shared memory for every row.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cb_shared.cuh"

namespace cb {

static __device__ uint32_t g_err_shared;
static std::atomic<bool> g_used_shared{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_shared() { return g_used_shared ? take_word(g_err_shared) : 0u; }

namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 128;
constexpr float kNone = -INFINITY;
// K and V in buffers of their own, loaded at once: 64 sequences of 8 heads over 4096 rows 97 us for heads of 128 (123
// with one buffer, V after the scores); of 256, where fewer CTAs then fit an SM, 201 (194).
template <int HD>
constexpr bool kBoth = HD <= 128;

// The pieces: first the prefix's (group, KV head, row tile, run of keys), then the own ones (sequence, KV
// head, row tile, run of keys).  Rows of a tile are consecutive (query, head of the KV head) pairs.
struct Pieces {
  int chunk, own_chunk;          // keys of a run (multiples of kKeys)
  int n_chunk, n_own;            // runs that a row's pieces are kept for: of the longest prefix, of the capacity
  int own_tiles;                 // row tiles of a sequence
  int first[kMaxGroups + 1];     // pieces before group g
  float* part;                   // [rows of q and heads][n_chunk + n_own][hd + 2]: o, m, l
};

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) k_shared_simt(const __grid_constant__ Shared p, const __grid_constant__ Pieces w) {
  constexpr int PAD = 4, LD = HD + PAD, PER = HD / 8;
  extern __shared__ float smem[];
  float* sq = smem;                          // [kRows][LD]
  float* sk = sq + kRows * LD;               // [kKeys][LD]
  float* sv = kBoth<HD> ? sk + kKeys * LD : sk;          // [kKeys][LD]
  float* sp = sv + kKeys * LD;               // [kRows][kKeys + PAD]
  __shared__ int s_last[kRows];
  const int tid = threadIdx.x, r = tid >> 3, c = tid & 7;
  pdl_wait();
  pdl_trigger();
  // ---- which piece
  int b = blockIdx.x;
  const bool own = b >= w.first[p.n_groups];
  int h, rt, run, n_rows, key0, keys;
  int64_t t0;                                // first query of the rows
  const T *k, *v;
  const int64_t W = (int64_t)p.Hkv * HD;
  if (!own) {
    int g = 0;
    while (b >= w.first[g + 1]) ++g;
    b -= w.first[g];
    const int runs = (p.len[g] + w.chunk - 1) / w.chunk;
    run = b % runs;
    b /= runs;
    t0 = (int64_t)p.seq0[g] * p.n_q;
    n_rows = (p.seq0[g + 1] - p.seq0[g]) * p.n_q * p.G;
    const int tiles = (n_rows + kRows - 1) / kRows;
    rt = b % tiles;
    h = b / tiles;
    key0 = run * w.chunk;
    keys = min(w.chunk, p.len[g] - key0);
    k = static_cast<const T*>(p.k) + (int64_t)p.row0[g] * W;
    v = static_cast<const T*>(p.v) + (int64_t)p.row0[g] * W;
  } else {
    b -= w.first[p.n_groups];
    run = b % w.n_own;
    b /= w.n_own;
    rt = b % w.own_tiles;
    b /= w.own_tiles;
    h = b % p.Hkv;
    const int s = b / p.Hkv;
    t0 = (int64_t)s * p.n_q;
    n_rows = p.n_q * p.G;
    key0 = run * w.own_chunk;
    keys = w.own_chunk;
    k = static_cast<const T*>(p.own_k) + (int64_t)s * p.capacity * W;
    v = static_cast<const T*>(p.own_v) + (int64_t)s * p.capacity * W;
  }
  const int row = rt * kRows + r;            // of the group or sequence
  const bool on = row < n_rows;
  const int64_t t = t0 + (on ? row / p.G : 0);
  const int64_t qrow = t * p.H + (int64_t)h * p.G + (on ? row % p.G : 0);
  if (c == 0) {
    const int l = on ? p.last[t] : -2;
    if (l < -2 || l >= p.capacity) atomicOr(&g_err_shared, ERRBIT_INDEX);
    s_last[r] = on ? shared_last(p, t) : -2;
  }
  __syncthreads();
  // the last key of this piece that a row sees, and that any does
  const int seen = own ? s_last[r] - key0 : (s_last[r] >= -1 ? keys - 1 : -1);
  if (own) {
    int mx = -1;
    for (int i = 0; i < kRows; ++i) mx = max(mx, s_last[i] - key0 + 1);
    keys = min(keys, mx);
  }
  float* part = w.part + (qrow * (w.n_chunk + w.n_own) + (own ? w.n_chunk : 0) + run) * (HD + 2);
  if (keys <= 0) {
    if (on && c == 0) {
      part[HD] = kNone;
      part[HD + 1] = 0.f;
    }
    return;
  }
  const float* qr = sq + r * LD;
  for (int i = c * 4; i < HD; i += 32) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) ld4(static_cast<const T*>(p.q) + qrow * HD + i, f);
    *reinterpret_cast<float4*>(sq + r * LD + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
  float m = kNone, l = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < keys; j0 += kKeys) {
    __syncthreads();
    auto rows_of = [&](auto with_k, auto with_v) {       // keys past the last one that is seen are not read
      for (int i = tid; i < kKeys * (HD / 4); i += kThreads) {
        const int j = i / (HD / 4), at = i % (HD / 4) * 4;
        float f[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
        if (j0 + j < keys) {
          const int64_t from = (int64_t)(key0 + j0 + j) * W + h * HD + at;
          if (with_k) ld4(k + from, f);
          if (with_v) ld4(v + from, e);
        }
        if (with_k) *reinterpret_cast<float4*>(sk + j * LD + at) = make_float4(f[0], f[1], f[2], f[3]);
        if (with_v) *reinterpret_cast<float4*>(sv + j * LD + at) = make_float4(e[0], e[1], e[2], e[3]);
      }
    };
    rows_of(std::true_type{}, std::bool_constant<kBoth<HD>>{});
    __syncthreads();
    // scores of keys c, c + 8, c + 16, c + 24
    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < HD; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(qr + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 x = *reinterpret_cast<const float4*>(sk + (c + 8 * q) * LD + i);
        z[q] = fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, z[q]))));
      }
    }
    float mx = m;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      z[q] = j0 + c + 8 * q <= seen ? z[q] * p.scale_log2 : -INFINITY;
      mx = fmaxf(mx, z[q]);
    }
#pragma unroll
    for (int i = 1; i < 8; i <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    const float keep = m == kNone ? 0.f : exp2f(m - mx);
    l *= keep;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] *= keep;
    m = mx;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float e = z[q] == -INFINITY ? 0.f : exp2f(z[q] - m);
      l += e;
      sp[r * (kKeys + PAD) + c + 8 * q] = e;
    }
    if (!kBoth<HD>) {
      __syncthreads();
      rows_of(std::false_type{}, std::true_type{});
      __syncthreads();
    }
    __syncwarp();                            // (a row's weights are its warp's)
#pragma unroll 4
    for (int j = 0; j < kKeys; ++j) {
      const float e = sp[r * (kKeys + PAD) + j];
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(sv + j * LD + i * 8 + c * 4);
        o[i] = fmaf(e, x.x, o[i]);
        o[i + 1] = fmaf(e, x.y, o[i + 1]);
        o[i + 2] = fmaf(e, x.z, o[i + 2]);
        o[i + 3] = fmaf(e, x.w, o[i + 3]);
      }
    }
  }
#pragma unroll
  for (int i = 1; i < 8; i <<= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  if (!on) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) part[(i / 4) * 32 + c * 4 + i % 4] = o[i];
  if (c == 0) {
    part[HD] = isnan(l) ? l : m;             // (a NaN's scores leave no maximum; the row is not to look empty)
    part[HD + 1] = l;
  }
}

// one warp per row and head
template <typename T, int HD>
__global__ void __launch_bounds__(256) k_shared_join_simt(const __grid_constant__ Shared p, const __grid_constant__ Pieces w) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= (int64_t)p.n_seq * p.n_q * p.H) return;
  const int64_t t = row / p.H;
  const int s = (int)(t / p.n_q), last = shared_last(p, t);
  int g = 0;
  while (s >= p.seq0[g + 1]) ++g;
  const int a = last >= -1 ? (p.len[g] + w.chunk - 1) / w.chunk : 0, b = last >= 0 ? last / w.own_chunk + 1 : 0;
  const float* part = w.part + row * (w.n_chunk + w.n_own) * (HD + 2);
  auto piece = [&](int i) { return part + (int64_t)(i < a ? i : w.n_chunk + i - a) * (HD + 2); };
  // sixteen (eight) pieces at a time, statistics and rows in one go, each batch joined to what came before it (one
  // piece after the other 6 x 3 queries of 4 heads over 1000 rows took 29 us)
  constexpr int PER = HD / 32, BATCH = PER <= 4 ? 16 : 8;
  float M = kNone, L = 0.f, o[PER];
#pragma unroll
  for (int q = 0; q < PER; ++q) o[q] = 0.f;
  for (int i0 = 0; i0 < a + b; i0 += BATCH) {
    float x[BATCH][PER], m = kNone, l = 0.f;
    if (lane < BATCH && i0 + lane < a + b) {
      m = piece(i0 + lane)[HD];
      l = piece(i0 + lane)[HD + 1];
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < a + b)
#pragma unroll
        for (int q = 0; q < PER; ++q) x[i][q] = piece(i0 + i)[q * 32 + lane];
    const float top = fmaxf(M, warp_max(m)), keep = M == kNone ? 0.f : exp2f(M - top);
    const float f = m == kNone ? 0.f : exp2f(m - top);                   // (a NaN is no infinity)
    L = fmaf(l, f, L * keep);
#pragma unroll
    for (int q = 0; q < PER; ++q) o[q] *= keep;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (i0 + i < a + b && fi != 0.f) o[q] = fmaf(x[i][q], fi, o[q]);
    }
    M = top;
  }
  L = warp_sum(L);
  const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
  for (int q = 0; q < PER; ++q) static_cast<T*>(p.out)[row * HD + q * 32 + lane] = from_f<T>(o[q] * inv);
}

// Runs of keys long enough that every piece is worth its start, and short enough that there are some for
// every SM.  False: more pieces than a grid holds.
bool cut(const Shared& p, Pieces* w) {
  const int64_t sms = 152;
  int64_t tiles = 0, longest = 0;
  for (int g = 0; g < p.n_groups; ++g) {
    tiles += ((int64_t)(p.seq0[g + 1] - p.seq0[g]) * p.n_q * p.G + kRows - 1) / kRows * p.Hkv;
    longest = std::max<int64_t>(longest, p.len[g]);
  }
  auto run = [&](int64_t keys, int64_t t) {
    const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(64, 4 * sms / std::max<int64_t>(t, 1)));
    return (int)std::max<int64_t>(kKeys, ((keys + pieces - 1) / pieces + kKeys - 1) / kKeys * kKeys);
  };
  w->chunk = run(longest, tiles);
  w->n_chunk = (int)((longest + w->chunk - 1) / w->chunk);
  int64_t at = 0;
  for (int g = 0; g < p.n_groups; ++g) {
    w->first[g] = (int)at;
    const int64_t rows = (int64_t)(p.seq0[g + 1] - p.seq0[g]) * p.n_q * p.G;
    at += (rows + kRows - 1) / kRows * p.Hkv * ((p.len[g] + w->chunk - 1) / w->chunk);
    if (at > INT32_MAX) return false;
  }
  w->first[p.n_groups] = (int)at;
  const int64_t own_tiles = ((int64_t)p.n_q * p.G + kRows - 1) / kRows;
  w->own_tiles = (int)own_tiles;
  w->own_chunk = run(p.capacity, own_tiles * p.Hkv * p.n_seq);
  w->n_own = (int)((p.capacity + w->own_chunk - 1) / w->own_chunk);
  return at + (double)own_tiles * p.Hkv * p.n_seq * w->n_own <= (double)INT32_MAX &&
         (double)p.n_seq * p.n_q * p.H / 8 <= (double)INT32_MAX;
}

template <typename T, int HD>
cudaError_t launch_hd(const Shared& p, const Pieces& w, cudaStream_t s) {
  const int64_t n = w.first[p.n_groups] + (int64_t)w.own_tiles * p.Hkv * p.n_seq * w.n_own;
  const size_t smem = ((kRows + (kBoth<HD> ? 2 : 1) * kKeys) * (HD + 4) + kRows * (kKeys + 4)) * sizeof(float);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_shared_simt<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  if (n > 0) {
    const cudaError_t e = launch_k(k_shared_simt<T, HD>, dim3((unsigned)n), dim3(kThreads), smem, s, p, w);
    if (e != cudaSuccess) return e;
  }
  const int64_t rows = (int64_t)p.n_seq * p.n_q * p.H;
  return launch_k(k_shared_join_simt<T, HD>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, p, w);
}
template <typename T>
cudaError_t launch_t(const Shared& p, const Pieces& w, cudaStream_t s) {
  switch (p.hd) {
    case 32: return launch_hd<T, 32>(p, w, s);
    case 64: return launch_hd<T, 64>(p, w, s);
    case 96: return launch_hd<T, 96>(p, w, s);
    case 128: return launch_hd<T, 128>(p, w, s);
    case 160: return launch_hd<T, 160>(p, w, s);
    case 192: return launch_hd<T, 192>(p, w, s);
    case 224: return launch_hd<T, 224>(p, w, s);
    case 256: return launch_hd<T, 256>(p, w, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// bytes of workspace; 0: too many pieces for one call
size_t shared_simt_ws_bytes(const Shared& p) {
  Pieces w;
  if (!cut(p, &w)) return 0;
  return (size_t)p.n_seq * p.n_q * p.H * (w.n_chunk + w.n_own) * (p.hd + 2) * sizeof(float) + 16;
}

cudaError_t launch_shared_simt(int dt, const Shared& p, void* ws, cudaStream_t s) {
  g_used_shared = true;
  Pieces w;
  if (!cut(p, &w)) return cudaErrorInvalidValue;
  w.part = static_cast<float*>(ws);
  return dt == DT_BF16 ? launch_t<bf16>(p, w, s) : launch_t<float>(p, w, s);
}

}  // namespace cb
