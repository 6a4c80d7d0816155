// Attention of a batch over a shared prefix on the tensor cores (bf16, head_dim 64 or 128); the mathematics
// is cb_shared.cu's: pieces with a running softmax, joined at the end.  Three kernels:
//
//   k_shared_prefix  the prefixes.  All rows (query, head) of a group's batch that share a KV head are rows of
//                    one matrix: S = Q K^T and O = P V by tcgen05.mma over 128-row and 128-key tiles, so that
//                    a prefix is read once per 128 rows.  Few rows are bound by the prefix's bytes (32 x 4 queries
//                    of 40 heads over 26600 rows in four prefixes: 6.1 TB/s), many by the chain from S over P to
//                    O: 0.94 us for a key tile on an SM, of which the products at the rate of a large matrix
//                    product are 0.67.
//   k_shared_own     each sequence's own rows: few rows, few keys, bound by the caches' bytes (the same 32 sequences
//                    of some 350 rows: 4.6 TB/s alone).
//   k_shared_join    joins a row's pieces: 1 us for few rows, 11 for 768 queries of 56 heads.
//
// Both of the first cut their work as one line of equal steps (key tiles of a (KV head, row tile); 16 keys of
// a (sequence, head)) into equal runs, one per worker, wherever a tile's end falls: with whole tiles per CTA a
// 4096-row prefix of 32 heads leaves a third of the 152 SMs idle.  A worker leaves one piece for every tile
// that its run touches, in slot worker + tile (along the line one of the two goes up at every new pair).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "cb_shared.cuh"
#include "cb_tc.cuh"

namespace cb {

static __device__ uint32_t g_err_shared_tc;
static std::atomic<bool> g_used_shared_tc{false};   // a kernel of this file was launched (or captured)

uint32_t take_error_shared_tc() { return g_used_shared_tc ? take_word(g_err_shared_tc) : 0u; }

namespace {

using tc::f2_add;
using tc::f2_fma;
using tc::f2_pack;
using tc::f2_unpack;
using tc::fmax3;

constexpr int BM = 128;              // rows of a tile
constexpr int BN = 128;              // keys of a tile
constexpr int SLAB = 128 * 128;      // bytes of one [128 rows x 64 elements] swizzled slab
constexpr int THREADS = 384;         // of the prefix kernel: copies and products, two groups of softmax
constexpr int kRegsIssue = 40, kRegsSoftmax = 232;      // registers a thread after the split; 40 + 2 x 232 = 3 x 168 as launched
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_O = 2 * BN;    // TMEM: S_0 | S_1 | O_0 | O_1
constexpr float kLazy = 8.0f;        // weights up to 2^8 before a row's maximum is raised
constexpr int kWorkers = 152;        // of the prefix kernel, one CTA per SM
constexpr int kOwnWarps = 4, kOwnThreads = 32 * kOwnWarps, kOwnCtas = 304;   // of the own rows' kernel
constexpr int TILE = 8;              // rows of its tiles
constexpr int kHeld = 2048;          // (sequence, row tile) pairs whose steps a CTA keeps in shared memory

struct Tc {
  Shared s;
  int total, workers;            // key tiles of all prefixes, the runs that they are cut into
  int ctas;                      // that take these runs by turns
  int first[kMaxGroups + 1];     // key tiles before group g
  int prob[kMaxGroups + 1];      // (KV head, row tile) pairs before group g
  int qpt;                       // queries of a row tile: 128 / G
  int slot_rows;                 // rows that a slot holds
  float* part;                   // [workers + pairs][slot_rows][hd], then m and l: see slot()
  // wide: the line holds row tiles with queries of one sequence, which go on from the prefix to the sequence's own
  // rows; or (split) to the own rows alone, and behind them the row tiles of the groups with the prefixes
  bool wide, split;
  int chunks;                    // row tiles of a sequence
  // own rows, where they have a kernel of their own
  int row_tiles;                 // of a sequence
  int own_slot_rows;
  int own_ctas;                  // CTAs of its kernel
  bool alone;                    // no prefix kernel runs before
  int32_t* plan;                 // [n_seq row_tiles + 1] steps before each, times Hkv; wide: how many row tiles are
                                 // live, their key tiles, [row tiles] the place of each among them (-1: none of
                                 // its queries sees anything), [live + 1] key tiles before each
  float* own_part;               // [workers + n_seq row_tiles Hkv][rows][hd], m, l
};

// the runs of a wide call's key tiles: a tile for each group of warps
__device__ __forceinline__ int wide_workers(int total, int workers) { return min(workers, (total + 1) / 2); }
__device__ __forceinline__ int row_tiles_of(const Tc& w, int g) {
  return ((w.s.seq0[g + 1] - w.s.seq0[g]) * w.s.n_q + w.qpt - 1) / w.qpt;
}
__device__ __forceinline__ float* slot(float* part, int rows, int hd, int worker, int pair) {
  return part + ((int64_t)worker + pair) * (rows * (hd + 2));
}

// A run's part inside one (KV head, row tile).
struct Seg {
  int h, pair;
  int tile, n;                   // its first key tile, and how many there are
  int end;                       // where it ends on the line
  int tok, queries;              // the row tile's first query, and how many there are
  int row0, len;                 // the prefix
  int own_tile, own_row, own_len;    // the first key tile of own rows, the first own row, how many are seen
};
constexpr int kWideTiles = 2048;     // row tiles of a wide call
// Rows of a sequence and KV head from which its own keys go with the prefixes' (split) if they do not fill tiles: the
// other kernel reads them once per 8 rows.  16 and 64 sequences over 4096 rows of 32 heads: 8 rows 38 and 97 us (27 and
// 72 apart), 16 rows 51 and 131 (52 and 185), 88 rows 124 (649).
constexpr int kSplitRows = 16;
struct Wide {                        // the live row tiles of a wide call, in order
  int first[kWideTiles + 1];         // key tiles before each; at the end those of one head
  int id[kWideTiles], last[kWideTiles];
  int n;
};
template <bool WIDE>
__device__ __forceinline__ Seg segment(const Tc& w, const Wide& wide, int i, int b) {
  const Shared& p = w.s;
  Seg x;
  int kt;
  if constexpr (WIDE) {
    const int per = wide.first[wide.n];
    x.h = i / per;
    int at = i - x.h * per, lo = 0, hi = wide.n - 1;         // the last one that starts at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (wide.first[mid] <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int id = wide.id[lo], of_seq = p.n_seq * w.chunks;
    kt = wide.first[lo + 1] - wide.first[lo];
    x.tile = at - wide.first[lo];
    x.pair = x.h * wide.n + lo;
    int g = 0;
    if (id < of_seq) {
      const int s = id / w.chunks, c = id - s * w.chunks;
      while (s >= p.seq0[g + 1]) ++g;
      x.tok = s * p.n_q + c * w.qpt;
      x.queries = min(w.qpt, p.n_q - c * w.qpt);
      x.len = w.split ? 0 : p.len[g];
      x.own_tile = (x.len + BN - 1) / BN;
      x.own_row = (int)(s * p.capacity);
      x.own_len = wide.last[lo] + 1;
    } else {
      while (id - of_seq >= w.prob[g + 1]) ++g;
      const int q0 = (id - of_seq - w.prob[g]) * w.qpt;
      x.tok = p.seq0[g] * p.n_q + q0;
      x.queries = min(w.qpt, (p.seq0[g + 1] - p.seq0[g]) * p.n_q - q0);
      x.len = p.len[g];
      x.own_tile = 0x7fffffff;
      x.own_row = x.own_len = 0;
    }
    x.row0 = p.row0[g];
  } else {
    int g = 0;
    while (i >= w.first[g + 1]) ++g;
    const int rts = row_tiles_of(w, g), at = i - w.first[g];
    kt = (p.len[g] + BN - 1) / BN;
    const int pl = at / kt;
    x.tile = at - pl * kt;
    x.h = pl / rts;
    x.pair = w.prob[g] + pl;
    const int q0 = (pl - x.h * rts) * w.qpt;
    x.tok = p.seq0[g] * p.n_q + q0;
    x.queries = min(w.qpt, (p.seq0[g + 1] - p.seq0[g]) * p.n_q - q0);
    x.row0 = p.row0[g];
    x.len = p.len[g];
    x.own_tile = 0x7fffffff;
    x.own_row = x.own_len = 0;
  }
  x.end = min(b, i + kt - x.tile);
  x.n = x.end - i;
  return x;
}
// keys of the segment's tile j that are there
template <bool WIDE>
__device__ __forceinline__ int keys_of(const Seg& x, int j) {
  return min(BN, WIDE && j >= x.own_tile ? x.own_len - (j - x.own_tile) * BN : x.len - j * BN);
}

// The row tiles of which some query sees something; the first CTA leaves them in the plan for the join.
__device__ __forceinline__ void make_wide(const Tc& w, Wide& wide, int tid, int threads) {
  const Shared& p = w.s;
  const int of_seq = p.n_seq * w.chunks, shared = w.split ? w.prob[p.n_groups] : 0, tiles = of_seq + shared;
  // The order of the row tiles.  Split: the groups' ones spread among the sequences', which are short and cost a start
  // and a piece each (all of these first, the CTAs that got them took three times as long as the others).
  auto id_at = [&](int i) -> int {
    const int a = i * shared / tiles, b = (i + 1) * shared / tiles;
    return b > a ? of_seq + a : i - a;
  };
  for (int pos = tid; pos < tiles; pos += threads) {
    int mx = -2, g = 0, n;
    const int i = id_at(pos);
    if (i < of_seq) {
      const int s = i / w.chunks, c = i - s * w.chunks;
      for (int j = c * w.qpt; j < min(p.n_q, (c + 1) * w.qpt); ++j) mx = max(mx, shared_last(p, (int64_t)s * p.n_q + j));
      while (s >= p.seq0[g + 1]) ++g;
      n = mx >= -1 ? (w.split ? 0 : (p.len[g] + BN - 1) / BN) + (mx + BN) / BN : 0;
    } else {
      while (i - of_seq >= w.prob[g + 1]) ++g;
      n = (p.len[g] + BN - 1) / BN;
    }
    wide.id[pos] = n;
    wide.last[pos] = mx;
  }
  __syncthreads();
  if (tid < 32) {
    const bool write = blockIdx.x == 0;
    int at = 0, units = 0;
    for (int i0 = 0; i0 < tiles; i0 += 32) {
      const int i = i0 + tid, n = i < tiles ? wide.id[i] : 0, mx = i < tiles ? wide.last[i] : -2;
      const unsigned live = __ballot_sync(0xffffffffu, n > 0);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += y;
      }
      const int to = at + __popc(live & ((1u << tid) - 1));
      if (n > 0) {
        wide.first[to] = units + incl - n;
        wide.id[to] = id_at(i);
        wide.last[to] = mx;
      }
      if (write) {
        if (i < tiles) w.plan[2 + id_at(i)] = n > 0 ? to : -1;
        if (n > 0) w.plan[2 + tiles + to] = units + incl - n;
      }
      at += __popc(live);
      units += __shfl_sync(0xffffffffu, incl, 31);
      __syncwarp();
    }
    if (tid == 0) {
      wide.first[at] = units;
      wide.n = at;
      if (write) {
        w.plan[0] = at;
        w.plan[1] = units;
        w.plan[2 + tiles + at] = units;
      }
    }
  }
  __syncthreads();
}

template <int HD, bool WIDE>
struct Layout {
  static constexpr int T_BYTES = HD / 64 * SLAB;             // a tile of Q, K or V
  static constexpr int OFF_Q = 0;                            // [2], by turns
  static constexpr int OFF_K = 2 * T_BYTES;                  // [2 groups]
  static constexpr int OFF_V = OFF_K + 2 * T_BYTES;          // [2]
  static constexpr int OFF_X = OFF_V + 2 * T_BYTES;          // [2 groups][BM] row max, row sum
  static constexpr int OFF_BAR = OFF_X + 4 * BM * 4;
  static constexpr int OFF_WIDE = OFF_BAR + 128;
  static constexpr int END = OFF_WIDE + (WIDE ? (int)sizeof(Wide) : 0) + 1024;
  static constexpr int SMEM = END > tc::kWholeSm ? END : tc::kWholeSm;
  static_assert(SMEM <= 227 * 1024, "shared memory exceeds the per-block limit");
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Two groups take a segment's key tiles by turns.  A group is four warps of softmax, one thread per row of the tile
// with its 128 scores in registers, one warp that issues its copies and one that issues its products, so that the
// chain S -> softmax -> P V -> S of the group's next tile holds no copy and no wait for one.  K's buffer is refilled
// as soon as S is there, V's once P V is done, across the ends of segments; Q alternates between two buffers, which
// are also the way out of a segment's rows.  Warps whose 32 rows do not exist (few queries) leave the softmax to
// the others.
//
// WIDE: the calls with many queries of each sequence.  A row tile's queries are of one sequence and its key tiles go
// on from the prefix's to the sequence's own, under each row's bound, so that own rows need no kernel of their own;
// row tiles of padding are left out.  (8 questions of 48 to 96 queries of 56 heads over 16000 rows: 299 us without.)
// Where sequences do not fill their tiles the prefixes' tiles are packed from a whole group's queries and only the own
// keys' are a sequence's own (split: 29 of 88 queries of 32 heads over 8204 rows 332 us, 1787 with the own rows' kernel).
//
// Barriers of a group: K and V have landed, S and P V are done, P is written.  How far the segments' results have
// been read (from TMEM, and out of Q's buffer) is a count that the issuing warps look at: they may be ahead by more
// than a barrier's phase can tell.
__device__ __forceinline__ bool wait_count(const int* count, int n) {
  for (uint32_t i = 0; i < tc::kWaitLimit; ++i) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(tc::smem_u32(count)) : "memory");
    if (v >= n) return true;
  }
  return false;
}

template <int HD, bool WIDE>
__global__ void __launch_bounds__(THREADS, 1)
    k_shared_prefix(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmOwnK,
                    const __grid_constant__ CUtensorMap tmOwnV, const __grid_constant__ Tc w) {
  using L = Layout<HD, WIDE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  float* xm = reinterpret_cast<float*>(base + L::OFF_X);     // [2][BM] row max, then [2][BM] row sum
  float* xl = xm + 2 * BM;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::OFF_BAR);
  uint64_t* q_full = bars + 12;                              // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);
  int* read_out = reinterpret_cast<int*>(bars + 14) + 1;     // warps that have read out their part of a segment
  // (the warp's number from one lane: the compiler then knows it to be one for the warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int wg = warp >> 2, quad = warp & 3;
  // warps 0 and 3 copy, 1 and 2 issue products, for groups 0 and 1; then the groups' softmax
  const int grp = wg == 0 ? warp >> 1 : wg - 1;
  uint64_t* k_full = bars + 6 * grp;
  uint64_t* v_full = k_full + 1;
  uint64_t* s_full = k_full + 2;
  uint64_t* pv_done = k_full + 3;
  uint64_t* p_full = k_full + 4;                             // [2]: of the tile's first 64 keys, and of the others
  const Shared& p = w.s;
  Wide& wide = *reinterpret_cast<Wide*>(base + L::OFF_WIDE);

  if (tid == 0) {
    for (int i = 0; i < 14; ++i) tc::mbar_init(&bars[i], i < 12 && i % 6 >= 4 ? 4 : 1);
    *read_out = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  int total = w.total, workers = w.workers;
  if (!WIDE) pdl_wait();
  if (WIDE) {
    pdl_wait();
    make_wide(w, wide, tid, THREADS);
    total = wide.first[wide.n] * p.Hkv;
    workers = wide_workers(total, workers);
  }
  pdl_trigger();                   // (before TMEM is allocated: see tc::kWholeSm)
  if (WIDE && (int)blockIdx.x >= workers) return;
  int run = blockIdx.x, b = run_start(total, run + 1, workers);
  Seg cur = segment<WIDE>(w, wide, run_start(total, run, workers), b);
  auto next = [&]() -> bool {      // the segment behind cur: of its run, or of the CTA's next one
    int a = cur.end;
    if (a >= b) {
      run += gridDim.x;
      if (run >= workers) return false;
      a = run_start(total, run, workers);
      b = run_start(total, run + 1, workers);
    }
    cur = segment<WIDE>(w, wide, a, b);
    return true;
  };
  if (warp == 4) {
    tc::tmem_alloc(tmem_slot, TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint8_t* sK = base + L::OFF_K + grp * L::T_BYTES;
  uint8_t* sV = base + L::OFF_V + grp * L::T_BYTES;
  bool ok = true;                  // of this warp; the others of a segment find out by their own waits
  int u = 0;                       // the group's tiles so far: the phase of its barriers

  if (wg == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (quad == 0 || quad == 3) {
      // -------------------------------------------------------------- copies
      int nk = 0, nv = 0, nq = 0;
      for (int nseg = 0; ok; ++nseg) {
        if (grp == 0) {
          ok = nseg < 2 || __all_sync(0xffffffffu, wait_count(read_out, 8 * (nseg - 1)));
          if (!ok) break;
          ++nq;
          if (lane == 0) {
            uint64_t* bar = &q_full[nseg & 1];
            tc::mbar_expect_tx(bar, HD * 2 * p.G * w.qpt);
            for (int s = 0; s < HD / 64; ++s)
              tma_load_3d(base + L::OFF_Q + (nseg & 1) * L::T_BYTES + s * SLAB, &tmQ, bar, 64 * s, cur.h * p.G,
                          cur.tok);
          }
          __syncwarp();
        }
        const int col = cur.h * HD;
        for (int t = grp; t < cur.n; t += 2, ++u) {
          const int j = cur.tile + t;
          const bool own = WIDE && j >= cur.own_tile;
          const int row = own ? cur.own_row + (j - cur.own_tile) * BN : cur.row0 + j * BN;
          if (u > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(s_full, (u - 1) & 1));
          if (!ok) break;
          ++nk;
          if (lane == 0) {
            tc::mbar_expect_tx(k_full, L::T_BYTES);
            for (int s = 0; s < HD / 64; ++s) tc::tma_load_2d(sK + s * SLAB, own ? &tmOwnK : &tmK, k_full, col + 64 * s, row);
          }
          __syncwarp();
          if (u > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(pv_done, (u - 1) & 1));
          if (!ok) break;
          ++nv;
          if (lane == 0) {
            tc::mbar_expect_tx(v_full, L::T_BYTES);
            for (int s = 0; s < HD / 64; ++s) tc::tma_load_2d(sV + s * SLAB, own ? &tmOwnV : &tmV, v_full, col + 64 * s, row);
          }
          __syncwarp();
        }
        if (!ok || !next()) break;
      }
      if (!ok) {                   // give the copies in flight as long again before the memory is given up
        if (nk > 0) tc::mbar_wait(k_full, (nk - 1) & 1);
        if (nv > 0) tc::mbar_wait(v_full, (nv - 1) & 1);
        for (int i = max(0, nq - 2); i < nq; ++i) tc::mbar_wait(&q_full[i & 1], (i >> 1) & 1);
      }
    } else {
      // -------------------------------------------------------------- products
      constexpr uint32_t idesc_s = tc::idesc_bf16_f32(BM, BN), idesc_o = tc::idesc_bf16_f32(BM, HD, true);
      const uint64_t kd = tc::desc_sw128(tc::smem_u32(sK)), vd = tc::desc_sw128_mn(tc::smem_u32(sV), SLAB);
      const uint32_t tS = tmem + grp * BN, tO = tmem + TM_O + grp * HD;
      for (int nseg = 0; ok; ++nseg) {
        const uint64_t qd = tc::desc_sw128(tc::smem_u32(base + L::OFF_Q + (nseg & 1) * L::T_BYTES));
        for (int t = grp; t < cur.n; t += 2, ++u) {
          const int keys = keys_of<WIDE>(cur, cur.tile + t);
          // Q: a group that had no tile in segments of one may be here while the buffer still holds the segment's before
          // the last, and the barrier's phase cannot tell; once that has been read out it can.  S goes where P is, until
          // P V is done.
          ok = __all_sync(0xffffffffu, (t != grp || ((nseg < 2 || wait_count(read_out, 8 * (nseg - 1))) &&
                                                     tc::mbar_wait(&q_full[nseg & 1], (nseg >> 1) & 1))) &&
                                           tc::mbar_wait(k_full, u & 1) && (u == 0 || tc::mbar_wait(pv_done, (u - 1) & 1)));
          if (!ok) break;
          tc::tc_fence_after();
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
              const uint32_t off = ((k >> 2) * SLAB + (k & 3) * 32) >> 4;
              tc::mma_bf16(tS, qd + off, kd + off, idesc_s, k > 0);
            }
            tc::mma_commit(s_full);
          }
          __syncwarp();
          ok = __all_sync(0xffffffffu, tc::mbar_wait(v_full, u & 1));
          if (ok && keys < BN) {
            // what the copy brought from behind the prefix may be no number: times a weight of 0 it would stay none
            for (int c = lane; c < (BN - keys) * 8; c += 32)
#pragma unroll
              for (int s = 0; s < HD / 64; ++s)
                *reinterpret_cast<uint4*>(sV + s * SLAB + keys * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            tc::fence_proxy_async_smem();
            __syncwarp();
          }
          // the segment's first tile writes O, once the segment before has been read out
          ok = ok && __all_sync(0xffffffffu, t != grp || nseg == 0 || wait_count(read_out, 8 * nseg));
#pragma unroll
          for (int h = 0; h < 2; ++h) {            // (the second half of P is written while the first multiplies)
            ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(&p_full[h], u & 1));
            if (!ok) break;
            tc::tc_fence_after();
            if (tc::elect_one()) {
#pragma unroll
              for (int k = h * (BN / 32); k < (h + 1) * (BN / 32); ++k)
                tc::mma_bf16_ts(tO, tS + k * 8, vd + (uint64_t)((k * 16 * 128) >> 4), idesc_o, (t != grp || k > 0) ? 1u : 0u);
              if (h) tc::mma_commit(pv_done);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        if (!ok || !next()) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---------------------------------------------------------------- softmax
    const int r = quad * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = trow + grp * BN, tO = trow + TM_O + grp * HD;
    auto softmax_sync = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    for (int nseg = 0;; ++nseg) {
      const int turn = nseg & 1;   // Q's buffer
      const int rows = cur.queries * p.G;
      const bool work = quad * 32 < rows;
      const int mine = WIDE && r < rows ? shared_last(p, cur.tok + r / p.G) + 1 : 0;       // own rows that the row sees
      float m_used = -INFINITY, l = 0.f;
      for (int t = grp; t < cur.n; t += 2, ++u) {
        const int j = cur.tile + t;
        const int keys = WIDE && j >= cur.own_tile ? mine - (j - cur.own_tile) * BN : cur.len - j * BN;    // that the row sees
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(s_full, u & 1));
        if (work && ok) {
          uint32_t sr[BN];
          tc::tc_fence_after();
#pragma unroll
          for (int c = 0; c < BN; c += 32) tc::tmem_ld32_nowait(tS + c, sr + c);
          tc::tmem_wait_ld64(sr);
          tc::tmem_wait_ld64(sr + 64);
          if (__any_sync(0xffffffffu, keys < BN)) {
#pragma unroll
            for (int c = 0; c < BN; ++c)
              if (c >= keys) sr[c] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = -INFINITY;
#pragma unroll
          for (int c = 0; c < BN; c += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mx[q] = fmax3(mx[q], __uint_as_float(sr[c + 2 * q]), __uint_as_float(sr[c + 2 * q + 1]));
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
          if (t == grp) {
            m_used = mt;           // O_g is written, not added to, by this tile's P V
          } else {
            const bool need = mt > m_used + kLazy;
            if (__any_sync(0xffffffffu, need)) {               // (S was issued after the last P V had completed)
              const float alpha = need ? tc::ex2_approx(m_used - mt) : 1.0f;
#pragma unroll 1
              for (int c = 0; c < HD / 16; ++c) {
                float o[16];
                tc::tmem_ld16(tO + c * 16, o);
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] *= alpha;
                tc::tmem_st16(tO + c * 16, o);
              }
              l *= alpha;
              if (need) m_used = mt;
            }
          }
          const float off = m_used == -INFINITY ? 0.f : -m_used;
          const uint64_t f2 = f2_pack(p.scale_log2, p.scale_log2), o2 = f2_pack(off, off);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const int k0 = c * 32 + 2 * q;
              const float2 z = f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[k0]), __uint_as_float(sr[k0 + 1])), f2, o2));
              const float p0 = tc::ex2_approx(z.x), p1 = tc::ex2_approx(z.y);
              sum[q & 1] = f2_add(sum[q & 1], f2_pack(p0, p1));
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
              pk[q] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            tc::tmem_st16u_nowait(tS + c * 16, pk);
            if (c == 1) {
              tc::tmem_wait_st();
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(p_full);
            }
          }
          const float2 sm = f2_unpack(f2_add(sum[0], sum[1]));
          l += sm.x + sm.y;
          tc::tmem_wait_st();
          tc::tc_fence_before();
        } else if (lane == 0) {
          tc::mbar_arrive(p_full);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + 1);
      }
      // -------------------------------------------------------------- the segment's piece
      // both groups' row statistics meet in shared memory
      ok = ok && (grp >= cur.n || __all_sync(0xffffffffu, tc::mbar_wait(pv_done, (u - 1) & 1)));
      xm[grp * BM + r] = m_used;
      xl[grp * BM + r] = l;
      tc::tc_fence_before();
      softmax_sync();
      tc::tc_fence_after();
      if (ok && work) {            // (uniform over the warp: the loads from TMEM are the whole warp's)
        const float ma = xm[r], mb = xm[BM + r], mm = fmaxf(ma, mb);
        const float a0 = ma == -INFINITY ? 0.f : tc::ex2_approx(ma - mm);
        const float a1 = mb == -INFINITY ? 0.f : tc::ex2_approx(mb - mm);
        // (a sum that is no number counts even though no maximum was found beside it)
        const float lt = (ma == -INFINITY ? xl[r] : xl[r] * a0) + (mb == -INFINITY ? xl[BM + r] : xl[BM + r] * a1);
        float* out = slot(w.part, w.slot_rows, HD, run, cur.pair);
        if (grp == 0 && r < rows) {
          out[w.slot_rows * HD + r] = isnan(lt) ? lt : mm;
          out[w.slot_rows * (HD + 1) + r] = lt;
        }
        // The rows leave through Q's buffer, HD / 4 columns of the warp's 32 rows at a time, so that a store
        // covers whole lines (each thread storing its own row took 2.1 us for 126 rows).
        constexpr int C4 = HD / 16;  // 16-byte words of a row's part
        uint8_t* st = base + L::OFF_Q + turn * L::T_BYTES + (grp * 4 + quad) * (32 * C4 * 16);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int col = grp * (HD / 2) + c * (HD / 4);
#pragma unroll
          for (int h = 0; h < C4 / 4; ++h) {
            float o0[16], o1[16];
            tc::tmem_ld16(trow + TM_O + col + h * 16, o0);
            if (cur.n > 1) {       // (else O_1 was never written)
              tc::tmem_ld16(trow + TM_O + HD + col + h * 16, o1);
            } else {
#pragma unroll
              for (int q = 0; q < 16; ++q) o1[q] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) o0[q] = o0[q] * a0 + o1[q] * a1;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4*>(st + lane * (C4 * 16) + (((h * 4 + q) ^ (lane & (C4 - 1))) << 4)) =
                  make_float4(o0[4 * q], o0[4 * q + 1], o0[4 * q + 2], o0[4 * q + 3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C4; ++i) {
            const int rr = i * (32 / C4) + lane / C4, q = lane & (C4 - 1), row = quad * 32 + rr;
            if (row < rows)
              *reinterpret_cast<float4*>(out + (int64_t)row * HD + col + q * 4) =
                  *reinterpret_cast<const float4*>(st + rr * (C4 * 16) + ((q ^ (rr & (C4 - 1))) << 4));
          }
          __syncwarp();
        }
        tc::fence_proxy_async_smem();            // (before Q comes into the same place)
      }
      tc::tc_fence_before();
      softmax_sync();              // the statistics are free
      if (lane == 0) {
        __threadfence_block();
        atomicAdd(read_out, 1);
      }
      if (!next()) break;          // (uniform)
    }
  }
  if (!ok && lane == 0) atomicOr(&g_err_shared_tc, ERRBIT_TIMEOUT);
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---- own rows ---------------------------------------------------------------------------------
// A step is 16 KW keys of one (sequence, KV head): 8 KB of K and V, by TMA into the warp's own stages, three in
// flight.  The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with the keys (then the channels)
// as the 16 rows of mma.m16n8k16 and up to 8 query rows as its columns: a token's few rows fill the
// instruction.  Every warp is a worker with an equal run of the line of steps and meets no other.
template <int HD>
struct Own {
  static constexpr int KW = 128 / HD, KT = 16 * KW;
  static constexpr int HALF = KT * HD * 2;                   // bytes of K (or V) of a step
  static constexpr int NST = 3;
  static constexpr int OFF_BAR = kOwnWarps * NST * 2 * HALF;
  static constexpr int SMEM = OFF_BAR + kOwnWarps * NST * 8 + kOwnThreads * 8 + kHeld * 4 + 1024;
};

__device__ __forceinline__ void mma_bf16_16x8(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t* a, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t* a, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
// 8 x 8 transposition of 16-bit pairs across the warp
__device__ __forceinline__ uint32_t transpose_pairs(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A (sequence, row tile, head) counts this many steps more on the line than it has: its start and its piece cost
// a worker about as much.
constexpr int kUnitCost = 1;
// how many workers share the line: a run has two steps at least
__device__ __forceinline__ int own_workers(int total, int workers) { return max(1, min(workers, total / 2)); }

template <int HD>
__global__ void __launch_bounds__(kOwnThreads, 2)
    k_shared_own(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Tc w) {
  using L = Own<HD>;
  constexpr int KS = HD / 16, SLABS = HD / 64, SL = L::KT * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  const Shared& p = w.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* stages = base + warp * L::NST * 2 * L::HALF;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + L::OFF_BAR) + warp * L::NST;
  int2* before = reinterpret_cast<int2*>(base + L::OFF_BAR + kOwnWarps * L::NST * 8);
  int* held = reinterpret_cast<int*>(before + kOwnThreads);      // [min(entries, kHeld)] steps
  const int R = p.n_q * p.G, entries = p.n_seq * w.row_tiles;
  if (lane == 0) {
    for (int i = 0; i < L::NST; ++i) tc::mbar_init(&full[i], 1);
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  // Nothing here needs the prefix kernel's results, only that everything before it is done, which that
  // kernel has seen before it let this one start; the wait at the end makes this one end after it.
  if (w.alone) pdl_wait();
  pdl_trigger();
  // ---- where this worker's run lies: thread i sums the steps of a share of the entries (sequence, row tile),
  // a scan places them; the first CTA writes the plan for the join
  auto row_last = [&](int e, int r) -> int {             // -1: no own row
    const int s = e / w.row_tiles, row = (e - s * w.row_tiles) * TILE + r;
    return r >= TILE || row >= R ? -1 : max(-1, shared_last(p, (int64_t)s * p.n_q + row / p.G));
  };
  auto count_steps = [&](int e) -> int {
    const int s = e / w.row_tiles, row0 = (e - s * w.row_tiles) * TILE;
    int mx = -1;
    for (int j = row0 / p.G; j <= (min(R, row0 + TILE) - 1) / p.G; ++j) mx = max(mx, shared_last(p, (int64_t)s * p.n_q + j));
    return (mx + L::KT) / L::KT;
  };
  auto steps_of = [&](int e) -> int { return e < kHeld ? held[e] : count_steps(e); };
  auto on_line = [&](int n) -> int { return n > 0 ? (n + kUnitCost) * p.Hkv : 0; };
  const int share = (entries + kOwnThreads - 1) / kOwnThreads, e0 = min(entries, tid * share), e1 = min(entries, e0 + share);
  int mine = 0, steps = 0;                               // on the line, and steps
  for (int e = e0; e < e1; ++e) {
    const int n = count_steps(e);
    if (e < kHeld) held[e] = n;
    mine += on_line(n);
    steps += n * p.Hkv;
  }
  int incl = mine, incl_steps = steps;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, incl_steps, o);
    if (lane >= o) {
      incl += y;
      incl_steps += z;
    }
  }
  __shared__ int2 wsum[kOwnWarps];
  if (lane == 31) wsum[warp] = make_int2(incl, incl_steps);
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int x = 0; x < kOwnWarps; ++x) {
    if (x < warp) {
      incl += wsum[x].x;
      incl_steps += wsum[x].y;
    }
    total += wsum[x].x;
  }
  before[tid] = make_int2(incl - mine, incl_steps - steps);
  if (blockIdx.x == 0) {
    int at = incl - mine;
    for (int e = e0; e < e1; ++e) {
      w.plan[e] = at;
      at += on_line(steps_of(e));
    }
    if (tid == 0) w.plan[entries] = total;
  }
  __syncthreads();
  struct Pos {
    int e, h, k, n;       // entry, head, step of the unit, steps in a unit of the entry
    int step;             // the step's number among all
  };
  // place x of the line: the first step at or behind it (x < total)
  auto place = [&](int x) -> Pos {
    // the last thread whose share starts at or before it and is not empty
    int c = 0;
    for (int i = lane; i < kOwnThreads; i += 32)
      if (before[i].x <= x && i * share < entries) c = i;
    c = __reduce_max_sync(0xffffffffu, c);
    int left = x - before[c].x, step = before[c].y;
    Pos r;
    for (int f = c * share;; f += 32) {
      const int n = f + lane < entries ? steps_of(f + lane) : 0, mine = on_line(n);
      int in = mine, st = n * p.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, in, o), z = __shfl_up_sync(0xffffffffu, st, o);
        if (lane >= o) {
          in += y;
          st += z;
        }
      }
      const unsigned hit = __ballot_sync(0xffffffffu, left < in);
      if (hit || f + 32 >= entries) {
        const int who = hit ? __ffs(hit) - 1 : 31;
        r.e = f + who;
        r.n = __shfl_sync(0xffffffffu, n, who);
        left -= __shfl_sync(0xffffffffu, in - mine, who);
        r.step = step + __shfl_sync(0xffffffffu, st - n * p.Hkv, who);
        break;
      }
      left -= __shfl_sync(0xffffffffu, in, 31);
      step += __shfl_sync(0xffffffffu, st, 31);
    }
    r.h = left / (r.n + kUnitCost);
    r.k = max(0, left - r.h * (r.n + kUnitCost) - kUnitCost);
    r.step += r.h * r.n + r.k;
    return r;
  };
  const int n_work = own_workers(total, gridDim.x * kOwnWarps), worker = warp * gridDim.x + blockIdx.x;
  if (worker < n_work && total > 0) {
    const int va = run_start(total, worker, n_work), vb = run_start(total, worker + 1, n_work);
    Pos cur = place(va);
    int b;
    if (vb < total) {
      b = place(vb).step;
    } else {
      b = 0;
#pragma unroll
      for (int x = 0; x < kOwnWarps; ++x) b += wsum[x].y;
    }
    const int a = cur.step;
    auto advance = [&](Pos& x) {
      if (++x.k < x.n) return;
      x.k = 0;
      if (++x.h < p.Hkv) return;
      x.h = 0;
      for (++x.e; x.e < entries; ++x.e)
        if ((x.n = (__reduce_max_sync(0xffffffffu, row_last(x.e, lane)) + L::KT) / L::KT) > 0) return;
    };
    auto fill = [&](const Pos& x, int st) {
      if (lane != 0) return;
      const int row = (int)((int64_t)(x.e / w.row_tiles) * p.capacity) + x.k * L::KT;
      tc::mbar_expect_tx(&full[st], 2 * L::HALF);
#pragma unroll
      for (int i = 0; i < SLABS; ++i) {
        tc::tma_load_2d(stages + st * 2 * L::HALF + i * SL, &tmK, &full[st], x.h * HD + 64 * i, row);
        tc::tma_load_2d(stages + st * 2 * L::HALF + L::HALF + i * SL, &tmV, &full[st], x.h * HD + 64 * i, row);
      }
    };
    Pos pre = cur;                                 // the next step to load
    int loaded = 0;
    for (; loaded < L::NST && a + loaded < b; ++loaded) {
      fill(pre, loaded);
      if (a + loaded + 1 < b) advance(pre);
    }
    // Q^T as the column operand: thread (g, t) holds row g, channels 2t, 2t + 1 (and 8 on) of every 16
    auto load_q = [&](const Pos& x, uint32_t (*qb)[2]) {
      const int s = x.e / w.row_tiles, row = (x.e - s * w.row_tiles) * TILE + g;
      const bool on = row < R;
      const int j = on ? row / p.G : 0;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(
          static_cast<const bf16*>(p.q) + (((int64_t)s * p.n_q + j) * p.H + (int64_t)x.h * p.G + (on ? row - j * p.G : 0)) * HD + 2 * t);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qb[k][0] = on ? q[k * 8] : 0u;
        qb[k][1] = on ? q[k * 8 + 4] : 0u;
      }
    };
    // a lane's row and 16-byte chunk in the matrices that ldmatrix reads: of K keys by channels, of V^T
    // channels by keys
    const int k_row = (lane & 7) + (lane & 8), k_chunk = lane >> 4;
    const int v_row = (lane & 7) + ((lane >> 4) << 3), v_chunk = (lane >> 3) & 1;
    bool ok = true;
    int done = 0;                                  // steps of the run
    uint32_t qb[KS][2], qn[KS][2];                 // this unit's queries, and the next one's
    int lv = row_last(cur.e, lane), lvn = lv;      // the last key of the tile's row `lane`, here and in the next unit
    if (a < b) load_q(cur, qb);
    while (ok && a + done < b) {
      // ---------------------------------------------------------------- a unit, or a part of one
      const int row0 = (cur.e % w.row_tiles) * TILE, nrow = min(TILE, R - row0);
      const int nk = __reduce_max_sync(0xffffffffu, lv) + 1;
      const int lastr[2] = {__shfl_sync(0xffffffffu, lv, 2 * t), __shfl_sync(0xffffffffu, lv, 2 * t + 1)};
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[KS][4];
#pragma unroll
      for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      const int n = min(cur.n - cur.k, b - a - done);
      Pos nx = cur;
      if (a + done + n < b) {
        nx.k = nx.n - 1;
        advance(nx);
        if (nx.e != cur.e) lvn = row_last(nx.e, lane);
        load_q(nx, qn);
      }
      for (int x = 0; x < n; ++x, ++done) {
        const int st = done % L::NST, key0 = (cur.k + x) * L::KT;
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(&full[st], (done / L::NST) & 1)))) break;
        uint8_t* sk = stages + st * 2 * L::HALF;
        uint8_t* sv = sk + L::HALF;
        if (nk - key0 < L::KT) {
          // rows behind the last one that is seen may hold anything
          for (int c = lane; c < (L::KT - (nk - key0)) * 8; c += 32)
#pragma unroll
            for (int i = 0; i < SLABS; ++i)
              *reinterpret_cast<uint4*>(sv + i * SL + (nk - key0) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();          // (before a copy into the same place)
          __syncwarp();
        }
#pragma unroll
        for (int kw = 0; kw < L::KW; ++kw) {
          float z[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t ka = tc::smem_u32(sk) + (kw * 16 + k_row) * 128;
#pragma unroll
          for (int k = 0; k < KS; k += 2) {        // two sums: the products of one wait for one another
            uint32_t f[4];
            int c = 2 * k + k_chunk;
            ldmatrix4(f, ka + (c >> 3) * SL + (((c & 7) ^ (k_row & 7)) << 4));
            mma_bf16_16x8(z, f, qb[k][0], qb[k][1]);
            c += 2;
            ldmatrix4(f, ka + (c >> 3) * SL + (((c & 7) ^ (k_row & 7)) << 4));
            mma_bf16_16x8(y, f, qb[k + 1][0], qb[k + 1][1]);
          }
          const int key = key0 + kw * 16 + g;
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = key + (i >> 1) * 8 <= lastr[i & 1] ? (z[i] + y[i]) * p.scale_log2 : -INFINITY;
          float mx0 = fmaxf(z[0], z[2]), mx1 = fmaxf(z[1], z[3]);
          if (__any_sync(0xffffffffu, mx0 > m[0] + kLazy || mx1 > m[1] + kLazy)) {
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) {
              mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, q));
              mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, q));
            }
            mx0 = fmaxf(mx0, m[0]);
            mx1 = fmaxf(mx1, m[1]);
            const float f0 = m[0] == -INFINITY ? 0.f : tc::ex2_approx(m[0] - mx0);
            const float f1 = m[1] == -INFINITY ? 0.f : tc::ex2_approx(m[1] - mx1);
            if (m[0] != -INFINITY) l[0] *= f0;     // (a NaN stays)
            if (m[1] != -INFINITY) l[1] *= f1;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[i][0] *= f0;
              o[i][1] *= f1;
              o[i][2] *= f0;
              o[i][3] *= f1;
            }
            m[0] = mx0;
            m[1] = mx1;
          }
          const float r0 = m[0] == -INFINITY ? 0.f : m[0], r1 = m[1] == -INFINITY ? 0.f : m[1];
          const float p0 = tc::ex2_approx(z[0] - r0), p1 = tc::ex2_approx(z[1] - r1), p2 = tc::ex2_approx(z[2] - r0),
                      p3 = tc::ex2_approx(z[3] - r1);
          l[0] += p0 + p2;
          l[1] += p1 + p3;
          const uint32_t b0 = transpose_pairs(pack_bf16(p0, p1)), b1 = transpose_pairs(pack_bf16(p2, p3));
          const uint32_t va = tc::smem_u32(sv) + (kw * 16 + v_row) * 128;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            uint32_t f[4];
            const int c = 2 * i + v_chunk;
            ldmatrix4_trans(f, va + (c >> 3) * SL + (((c & 7) ^ (v_row & 7)) << 4));
            mma_bf16_16x8(o[i], f, b0, b1);
          }
        }
        __syncwarp();
        if (a + loaded < b) {
          fill(pre, loaded % L::NST);
          ++loaded;
          if (a + loaded < b) advance(pre);
        }
      }
#pragma unroll
      for (int q = 4; q < 32; q <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], q);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], q);
      }
      float* out = slot(w.own_part, w.own_slot_rows, HD, worker, cur.e * p.Hkv + cur.h);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 2 * t + c;
        if (r >= nrow || !ok) continue;
        if (g == 0) {
          out[w.own_slot_rows * HD + r] = isnan(l[c]) ? l[c] : m[c];
          out[w.own_slot_rows * (HD + 1) + r] = l[c];
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          out[r * HD + i * 16 + g] = o[i][c];
          out[r * HD + i * 16 + 8 + g] = o[i][2 + c];
        }
      }
      cur = nx;
      lv = lvn;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qb[k][0] = qn[k][0];
        qb[k][1] = qn[k][1];
      }
    }
    if (!ok) {
      // report, and give the copies in flight as long again
      if (lane == 0) atomicOr(&g_err_shared_tc, ERRBIT_TIMEOUT);
      for (int i = max(0, loaded - L::NST); i < loaded; ++i) tc::mbar_wait(&full[i % L::NST], (i / L::NST) & 1);
    }
  }
  if (!w.alone) pdl_wait();
}

// ---- join: one warp per (query, head) ------------------------------------------------------------
// What does not come from the two kernels before is worked out before the wait for them.
template <int HD, bool WIDE>
__global__ void __launch_bounds__(256, WIDE ? 5 : 3) k_shared_join(const __grid_constant__ Tc w) {
  const Shared& p = w.s;
  const int t = blockIdx.x, hh = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int s = t / p.n_q, j = t - s * p.n_q, h = hh / p.G, gh = hh - h * p.G;
  const bool on = hh < p.H;
  // pieces of the prefix, then the own ones: slots are one worker apart
  int n_pre = 0, n_own = 0, r = 0;
  const float *pre = nullptr, *own = nullptr;
  const int64_t pre_step = (int64_t)w.slot_rows * (HD + 2), own_step = (int64_t)w.own_slot_rows * (HD + 2);
  if (!WIDE && on && w.total > 0) {
    int g = 0;
    while (s >= p.seq0[g + 1]) ++g;
    const int kt = (p.len[g] + BN - 1) / BN;
    if (kt > 0) {
      const int tl = t - p.seq0[g] * p.n_q, rt = tl / w.qpt, pl = h * row_tiles_of(w, g) + rt;
      const int x0 = w.first[g] + pl * kt, w0 = worker_of(w.total, x0, w.workers);
      n_pre = worker_of(w.total, x0 + kt - 1, w.workers) - w0 + 1;
      pre = slot(w.part, w.slot_rows, HD, w0, w.prob[g] + pl);
      r = (tl - rt * w.qpt) * p.G + gh;
    }
  }
  const int rr = j * p.G + gh, e = s * w.row_tiles + rr / TILE;
  // (the bounds were written before the call: the kernels that let this one start had waited for that)
  const bool only = !WIDE && w.alone && p.capacity == 0;
  if (only) pdl_wait();
  const int raw = p.last[t], last = shared_last(p, t);
  if (raw != last && hh == 0 && lane == 0) atomicOr(&g_err_shared_tc, ERRBIT_INDEX);
  if (!only) pdl_wait();
  pdl_trigger();
  if (!on) return;
  int r_own = rr % TILE;
  if (WIDE && last > -2) {
    const int of_seq = p.n_seq * w.chunks, tiles = of_seq + (w.split ? w.prob[p.n_groups] : 0), per = w.plan[1],
              total = per * p.Hkv, workers = wide_workers(total, w.workers);
    auto pieces = [&](int id, const float*& from) -> int {             // of a row tile
      const int li = w.plan[2 + id];
      if (li < 0) return 0;
      const int f = w.plan[2 + tiles + li], x0 = h * per + f, kt = w.plan[2 + tiles + li + 1] - f,
                w0 = worker_of(total, x0, workers);
      from = slot(w.part, w.slot_rows, HD, w0, h * w.plan[0] + li);
      return worker_of(total, x0 + kt - 1, workers) - w0 + 1;
    };
    const int c = j / w.qpt, at = (j - c * w.qpt) * p.G + gh;
    if (w.split) {
      int g = 0;
      while (s >= p.seq0[g + 1]) ++g;
      const int tl = t - p.seq0[g] * p.n_q, rt = tl / w.qpt;
      r = (tl - rt * w.qpt) * p.G + gh;
      n_pre = pieces(of_seq + w.prob[g] + rt, pre);
      r_own = at;
      if (last >= 0) n_own = pieces(s * w.chunks + c, own);
    } else {
      r = at;
      n_pre = pieces(s * w.chunks + c, pre);
    }
  }
  if (last == -2) n_pre = 0;
  if (!WIDE && last >= 0) {
    const int total = w.plan[p.n_seq * w.row_tiles], at = w.plan[e], n = (w.plan[e + 1] - at) / p.Hkv - kUnitCost;
    const int x0 = at + h * (n + kUnitCost) + kUnitCost;       // the unit's first step
    const int workers = own_workers(total, w.own_ctas * kOwnWarps), w0 = worker_of(total, x0, workers);
    n_own = worker_of(total, x0 + n - 1, workers) - w0 + 1;
    own = slot(w.own_part, w.own_slot_rows, HD, w0, e * p.Hkv + h);
  }
  const int n = n_pre + n_own;
  constexpr int PER = HD / 32;
  auto stat = [&](int i, int which) {
    return i < n_pre ? pre[i * pre_step + w.slot_rows * (HD + which) + r]
                     : own[(i - n_pre) * own_step + w.own_slot_rows * (HD + which) + r_own];
  };
  auto load = [&](int i, float* x) {
    const float* y = (i < n_pre ? pre + i * pre_step + r * HD : own + (i - n_pre) * own_step + r_own * HD) + lane * PER;
    if constexpr (PER == 4) {
      const float4 v = *reinterpret_cast<const float4*>(y);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(y);
      x[0] = v.x, x[1] = v.y;
    }
  };
  // Pieces come eight at a time, statistics and rows in one go (a row is mostly one batch, and the time of a
  // small join is that of its chain of loads), each batch joined to what came before it.
  constexpr int BATCH = WIDE ? 4 : 8;
  float M = -INFINITY, L = 0.f, o[PER];
#pragma unroll
  for (int c = 0; c < PER; ++c) o[c] = 0.f;
  for (int i0 = 0; i0 < n; i0 += BATCH) {
    float x[BATCH][PER], m = -INFINITY, l = 0.f;
    if (lane < BATCH && i0 + lane < n) {
      m = stat(i0 + lane, 0);
      l = stat(i0 + lane, 1);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < n) load(i0 + i, x[i]);
    const float top = fmaxf(M, warp_max(m)), keep = M == -INFINITY ? 0.f : tc::ex2_approx(M - top);
    const float f = m == -INFINITY ? 0.f : tc::ex2_approx(m - top);      // (a NaN is no infinity)
    L = fmaf(l, f, L * keep);
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] *= keep;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
      for (int c = 0; c < PER; ++c)
        if (i0 + i < n && fi != 0.f) o[c] = fmaf(x[i][c], fi, o[c]);
    }
    M = top;
  }
  L = warp_sum(L);
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  bf16* out = static_cast<bf16*>(p.out) + ((int64_t)t * p.H + hh) * HD + lane * PER;
  if constexpr (PER == 4) {
#pragma unroll
    for (int c = 0; c < PER; ++c) o[c] *= inv;
    st4(out, o);
  } else {
    *reinterpret_cast<uint32_t*>(out) = pack_bf16(o[0] * inv, o[1] * inv);
  }
}

// ---- host --------------------------------------------------------------------------------------
// How many runs of the line a CTA gets.  All CTAs' first runs come first on the line, so that the heads at work at one
// time are a part of all, and prefixes that several row tiles read come from L2 after the first.  29 x 88 queries of 32
// heads over 8204 rows 406 us with one run, 332 with two; 300 x 1 over 8192 180 and 171.  Two row tiles do not pay for
// the pieces (150 x 1 of 40 heads over 12267 128 and 141), nor do runs of 26 tiles (64 x 24 over 4096 166 and 180).
int slices(const Shared& s, const Tc& w, double tiles) {               // tiles of a CTA
  double again = 0;
  for (int g = 0; g < s.n_groups; ++g)
    if ((int64_t)(s.seq0[g + 1] - s.seq0[g]) * s.n_q > 2 * w.qpt) again += 4.0 * s.len[g] * s.Hkv * s.hd;
  return (int)std::max(1.0, std::min({ceil(again / 96e6), tiles / 40, 16.0}));
}

// what the kernels need beside the call itself; false: too much for one call
bool plan_tc(const Shared& s, Tc* w, size_t* bytes) {
  w->s = s;
  w->qpt = BM / s.G;
  w->chunks = (s.n_q + w->qpt - 1) / w->qpt;
  int64_t at = 0, pairs = 0, rows = 0;
  // Row tiles of one sequence each where they are not many more than tiles of a whole group's queries.
  int64_t packed = 0;
  for (int g = 0; g < s.n_groups; ++g) packed += ((int64_t)(s.seq0[g + 1] - s.seq0[g]) * s.n_q + w->qpt - 1) / w->qpt;
  const int64_t tiles = (int64_t)s.n_seq * w->chunks;
  // Where they are, own rows still go with the prefixes if a sequence's rows would read their keys several times over
  // in the other kernel.
  w->split = tiles + packed <= kWideTiles && 4 * tiles > 5 * packed && s.capacity > 0 && s.n_q * s.G >= kSplitRows;
  w->wide = w->split || (tiles <= kWideTiles && 4 * tiles <= 5 * packed);
  if (w->wide) {
    int64_t longest = 0, n = 0;
    for (int g = 0; g < s.n_groups; ++g) {
      longest = std::max<int64_t>(longest, s.len[g]);
      w->prob[g] = (int)n;                   // (split: row tiles before group g)
      if (w->split) n += ((int64_t)(s.seq0[g + 1] - s.seq0[g]) * s.n_q + w->qpt - 1) / w->qpt;
    }
    w->prob[s.n_groups] = (int)n;
    const int64_t tiles = (int64_t)s.n_seq * w->chunks + n;
    const double most = (double)tiles * s.Hkv * ((longest + BN - 1) / BN + (s.capacity + BN - 1) / BN);
    if (most > INT32_MAX / 2 || (s.H + 7) / 8 > 65535) return false;
    w->total = 0;
    w->ctas = (int)std::min<double>(kWorkers, std::max(1.0, (most + 1) / 2));
    w->workers = w->ctas * slices(s, *w, most / w->ctas);
    w->slot_rows = ((w->split ? w->qpt : std::min(s.n_q, w->qpt)) * s.G + 3) & ~3;
    w->own_slot_rows = w->slot_rows;
    w->alone = false;
    w->own_part = nullptr;
    w->row_tiles = 0;
    const size_t pre = (size_t)(w->workers + tiles * s.Hkv) * w->slot_rows * sizeof(float) * (s.hd + 2), at = (pre + 255) & ~size_t(255);
    w->part = nullptr;
    w->plan = reinterpret_cast<int32_t*>(at);
    *bytes = at + (2 * tiles + 3) * 4 + 16;
    return true;
  }
  for (int g = 0; g < s.n_groups; ++g) {
    w->first[g] = (int)at;
    w->prob[g] = (int)pairs;
    const int64_t queries = (int64_t)(s.seq0[g + 1] - s.seq0[g]) * s.n_q, kt = (s.len[g] + BN - 1) / BN;
    const int64_t n = kt ? (queries + w->qpt - 1) / w->qpt * s.Hkv : 0;
    at += n * kt;
    pairs += n;
    if (n) rows = std::max(rows, std::min<int64_t>(queries, w->qpt) * s.G);
    if (at > INT32_MAX / 2) return false;
  }
  w->first[s.n_groups] = (int)at;
  w->prob[s.n_groups] = (int)pairs;
  w->total = (int)at;
  w->ctas = (int)std::min<int64_t>(kWorkers, (at + 1) / 2);             // (a tile for each group of warps)
  w->own_ctas = kOwnCtas;
  if (at > 0 && s.capacity > 0) {
    // The own rows' kernel starts beside the prefixes', on SMs that are left to it, so that one's products and start
    // cover the other's bytes: as many as make both last alike, as far as the host can know (caches half full; a key
    // tile takes an SM 0.95 us of products or 1.3 of bytes, a CTA of the other kernel reads 32 GB/s and starts in 4 us).
    // 64 answers of 56 heads over 16384 rows 45.5 us, one kernel after the other 51.5; 4 of 32 over 4096 16.2 and 19.1.
    const double unit = (rows > 64 ? 0.95 : 1.3) * s.hd / 128, bytes = 2.0 * s.n_seq * s.capacity * s.Hkv * s.hd;
    double best = 1e30;
    int left = 4;
    for (int x = 4; x <= kWorkers / 2; x += 2) {
      const double t = std::max((double)at / (kWorkers - x) * unit + 4.0, bytes / (2 * x * 32e3) + 4.0);
      if (t < best) best = t, left = x;
    }
    w->ctas = std::min(w->ctas, kWorkers - left);
    w->own_ctas = 2 * left;
  }
  w->workers = w->ctas * slices(s, *w, (double)at / std::max(1, w->ctas));
  w->slot_rows = (int)((rows + 3) & ~3);
  w->row_tiles = (s.n_q * s.G + TILE - 1) / TILE;
  w->own_slot_rows = (std::min(TILE, s.n_q * s.G) + 3) & ~3;
  w->alone = at == 0;
  const double units = (double)s.n_seq * w->row_tiles * s.Hkv;
  if (s.capacity > 0 && units * ((s.capacity + 15) / 16 + kUnitCost) > (double)(INT32_MAX / 2)) return false;
  if ((s.H + 7) / 8 > 65535) return false;
  const size_t slot = sizeof(float) * (s.hd + 2);
  const size_t pre = at ? (size_t)(w->workers + pairs) * w->slot_rows * slot : 0;
  const size_t plan = s.capacity ? ((size_t)s.n_seq * w->row_tiles + 1) * 4 : 0;
  const size_t own = s.capacity ? (size_t)(kOwnCtas * kOwnWarps + units) * w->own_slot_rows * slot : 0;
  const size_t a = 0, b = (a + pre + 255) & ~size_t(255), c = (b + own + 255) & ~size_t(255);
  w->part = reinterpret_cast<float*>(a);
  w->own_part = reinterpret_cast<float*>(b);
  w->plan = reinterpret_cast<int32_t*>(c);
  *bytes = c + plan + 16;
  return true;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e == cudaSuccess && q == cudaDriverEntryPointSuccess) return reinterpret_cast<EncodeTiledFn>(p);
    if (e != cudaSuccess) cudaGetLastError();   // clears the error of this lookup only
    return static_cast<EncodeTiledFn>(nullptr);
  }();
  return fn;
}
// bf16, dims from the inside out without gaps, boxes of 64 elements, 128-byte swizzle
bool make_map(CUtensorMap* map, const void* ptr, std::initializer_list<int64_t> dims, std::initializer_list<int> box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3], one[3] = {1, 1, 1};
  int n = 0;
  for (int64_t x : dims) d[n++] = (cuuint64_t)x;
  n = 0;
  for (int x : box) bx[n++] = (cuuint32_t)x;
  st[0] = d[0] * 2;
  if (n == 3) st[1] = st[0] * d[1];
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n, const_cast<void*>(ptr), d, st, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_shared_mu;
uint32_t g_shared_attr[64];

template <int HD>
cudaError_t set_attrs() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> g(g_shared_mu);
  const uint32_t bit = HD == 128 ? 1u : 2u;
  if (dev >= 0 && dev < 64 && (g_shared_attr[dev] & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(k_shared_prefix<HD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD, false>::SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_shared_prefix<HD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD, true>::SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_shared_own<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Own<HD>::SMEM);
  if (e == cudaSuccess && dev >= 0 && dev < 64) g_shared_attr[dev] |= bit;
  return e;
}

template <int HD>
cudaError_t launch_hd(const Tc& w, cudaStream_t st) {
  const Shared& s = w.s;
  cudaError_t e = set_attrs<HD>();
  if (e != cudaSuccess) return e;
  const int64_t W = (int64_t)s.Hkv * HD;
  const dim3 join(s.n_seq * s.n_q, (s.H + 7) / 8);
  CUtensorMap q, k, v, own_k, own_v;
  if ((w.wide || w.total > 0) && !make_map(&q, s.q, {HD, s.H, (int64_t)s.n_seq * s.n_q}, {64, s.G, w.qpt})) return cudaErrorInvalidValue;
  if (w.wide) {
    // (what is not there is not read: any map will do)
    const bool pre = *std::max_element(s.len, s.len + s.n_groups) > 0, own = s.capacity > 0;
    const int64_t rows = s.n_seq * s.capacity;
    if ((pre && (!make_map(&k, s.k, {W, s.n_rows}, {64, BN}) || !make_map(&v, s.v, {W, s.n_rows}, {64, BN}))) ||
        (own && (!make_map(&own_k, s.own_k, {W, rows}, {64, BN}) || !make_map(&own_v, s.own_v, {W, rows}, {64, BN}))))
      return cudaErrorInvalidValue;
    if (!pre) k = v = q;
    if (!own) own_k = own_v = q;
    e = launch_k(k_shared_prefix<HD, true>, dim3(w.ctas), dim3(THREADS), Layout<HD, true>::SMEM, st, q, k, v, own_k, own_v, w);
    if (e != cudaSuccess) return e;
    return launch_k(k_shared_join<HD, true>, join, dim3(256), 0, st, w);
  }
  if (w.total > 0) {
    if (!make_map(&k, s.k, {W, s.n_rows}, {64, BN}) || !make_map(&v, s.v, {W, s.n_rows}, {64, BN})) return cudaErrorInvalidValue;
    e = launch_k(k_shared_prefix<HD, false>, dim3(w.ctas), dim3(THREADS), Layout<HD, false>::SMEM, st, q, k, v, k, v, w);
    if (e != cudaSuccess) return e;
  }
  if (s.capacity > 0) {
    const int64_t rows = s.n_seq * s.capacity;
    if (!make_map(&k, s.own_k, {W, rows}, {64, Own<HD>::KT}) || !make_map(&v, s.own_v, {W, rows}, {64, Own<HD>::KT}))
      return cudaErrorInvalidValue;
    e = launch_k(k_shared_own<HD>, dim3(w.own_ctas), dim3(kOwnThreads), Own<HD>::SMEM, st, k, v, w);
    if (e != cudaSuccess) return e;
  }
  return launch_k(k_shared_join<HD, false>, join, dim3(256), 0, st, w);
}

}  // namespace

bool shared_tc_taken(int dt, const Shared& p) { return dt == DT_BF16 && (p.hd == 64 || p.hd == 128) && p.G <= BM; }

// fn(part of the call, its first query), one after the other: with as many row tiles as a wide call takes, where the own
// keys are to go with the prefixes.
template <typename Fn>
static bool in_parts(const Shared& p, Fn fn) {
  const int64_t qpt = BM / p.G, chunks = (p.n_q + qpt - 1) / qpt, tiles = chunks * p.n_seq;
  int64_t packed = 0;
  for (int g = 0; g < p.n_groups; ++g) packed += ((int64_t)(p.seq0[g + 1] - p.seq0[g]) * p.n_q + qpt - 1) / qpt;
  if (p.capacity == 0 || (int64_t)p.n_q * p.G < kSplitRows ||
      (tiles <= kWideTiles && (4 * tiles <= 5 * packed || tiles + packed <= kWideTiles)))
    return fn(p, (int64_t)0);
  // whole sequences, or parts of one (twice the row tiles: the groups' ones count too)
  const int64_t seqs = std::max<int64_t>(1, kWideTiles / (2 * chunks)), queries = std::min<int64_t>(p.n_q, kWideTiles / 2 * qpt);
  const int64_t own = p.capacity * p.Hkv * p.hd * 2;
  for (int64_t s = 0; s < p.n_seq; s += seqs)
    for (int64_t j = 0; j < p.n_q; j += queries) {
      Shared x = p;
      x.n_seq = (int)std::min(seqs, p.n_seq - s);
      x.n_q = (int)std::min(queries, p.n_q - j);
      for (int g = 0; g <= p.n_groups; ++g) x.seq0[g] = (int32_t)std::min<int64_t>(std::max<int64_t>(p.seq0[g] - s, 0), x.n_seq);
      x.own_k = static_cast<const char*>(p.own_k) + s * own;
      x.own_v = static_cast<const char*>(p.own_v) + s * own;
      if (!fn(x, s * p.n_q + j)) return false;
    }
  return true;
}

size_t shared_tc_ws_bytes(const Shared& p) {
  size_t most = 0;
  const bool ok = in_parts(p, [&](const Shared& x, int64_t) {
    Tc w;
    size_t n;
    if (!plan_tc(x, &w, &n)) return false;
    most = std::max(most, n);
    return true;
  });
  return ok ? most : 0;
}

int shared_tc_launches(const Shared& p) {
  int launches = 0;
  in_parts(p, [&](const Shared& x, int64_t) {
    Tc w;
    size_t n;
    if (!plan_tc(x, &w, &n)) return false;
    launches += w.wide ? 2 : 1 + (w.total > 0 ? 1 : 0) + (x.capacity > 0 ? 1 : 0);
    return true;
  });
  return launches;
}

void reset_shared_tc_caches() {
  std::lock_guard<std::mutex> g(g_shared_mu);
  for (int i = 0; i < 64; ++i) g_shared_attr[i] = 0;
}

cudaError_t launch_shared_tc(const Shared& p, void* ws, cudaStream_t s) {
  g_used_shared_tc = true;
  cudaError_t e = cudaSuccess;
  in_parts(p, [&](const Shared& x, int64_t t0) {
    Tc w;
    size_t n;
    if (!plan_tc(x, &w, &n)) {
      e = cudaErrorInvalidValue;
      return false;
    }
    char* base = static_cast<char*>(ws);
    w.part = reinterpret_cast<float*>(base + reinterpret_cast<size_t>(w.part));
    w.own_part = reinterpret_cast<float*>(base + reinterpret_cast<size_t>(w.own_part));
    w.plan = reinterpret_cast<int32_t*>(base + reinterpret_cast<size_t>(w.plan));
    const int64_t row = (int64_t)p.H * p.hd * 2;
    w.s.q = static_cast<const char*>(p.q) + t0 * row;
    w.s.out = static_cast<char*>(p.out) + t0 * row;
    w.s.last = p.last + t0;
    e = p.hd == 128 ? launch_hd<128>(w, s) : launch_hd<64>(w, s);
    return e == cudaSuccess;
  });
  return e;
}

}  // namespace cb
