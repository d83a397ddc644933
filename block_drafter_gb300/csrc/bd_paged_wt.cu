// Accumulated attention weights (bd_paged_weights) on the tensor cores, for pages that make whole boxes.
//
// S^T = K Q^T with the slots on the MMA's M side: a thread owns one slot -- one TMEM lane -- and adds up
// its weights 2^(scale log2(e) s - log2(e) lse) over the columns, which are the rows, in a register.  So
// nothing crosses lanes, and a slot that holds anything at all touches its own lane only.
// The work is tiles of 128 slots of all requests.  A cluster takes every kth of them (one block where
// there are enough tiles; else its blocks share the KV heads and add their sums through distributed
// shared memory, in rank order) and passes, KV head by KV head, over the rows that see the tile, N at a
// time (as many whole tokens as fit): N = 16 for a token, 64 for a block, 128 for prompt rows, so that a call of few rows is bound by
// K's bytes, which stream through a ring across heads and tiles, and one of many rows by the
// exponentials and the tensor cores alike (a 128 x 128 tile: 512 cycles each on an SM).
//   warps 0-3, 4-7  take the row tiles in turn, each from its half of TMEM (N columns)
//   warp 8          issues the MMAs;  warp 9  brings K and Q by TMA
// Two blocks on an SM hide each other's start.  Measured: a token of each of 8 requests of up to 16 384
// slots 24.4 us, 5.0 TB/s; 64 rows of 2 requests through a window of 4096 12.6 us, half of it the start: list, page ids
// and first tiles.
#include "bd_paged_tc.cuh"

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_wt)

namespace {

constexpr int kThreads = 320;
constexpr int kMaxBlocks = 8;  // of a cluster

template <int D, int N> struct Wt {
  static constexpr int kKSlots = N == 16 ? 3 : N == 64 ? 2 : 1, kQSlots = 2;  // tiles of K, of rows
  static constexpr uint32_t kK = (D / 64) * kAtom, kQAtom = N * 128, kQ = (D / 64) * kQAtom;
  static constexpr uint32_t kOffQ = kKSlots * kK;
  static constexpr uint32_t kOffLse = kOffQ + kQSlots * kQ;  // [2 halves][2 turns][N] floats
  static constexpr uint32_t kOffSum = kOffLse + 16 * N;      // [2 tiles][2 halves][128] floats
  static constexpr uint32_t kOffList = kOffSum + 2048;       // tiles before each request
  static constexpr uint32_t kOffBar = kOffList + (BD_PAGED_MAX_REQUESTS + 2) * 4;
  // More than a third of an SM's shared memory: at most two blocks share an SM, so their TMEM always
  // fits.  Blocks of two calls on two streams that waited for TMEM there could wait for each other's clusters.
  static constexpr size_t kNeed = 1024 + kOffBar + 256, kSmem = kNeed > 78 * 1024 ? kNeed : 78 * 1024;
  static constexpr uint32_t kCols = 2 * N;
  static_assert(2 * kCols <= 512, "two blocks' TMEM");
};
struct WeightMaps {
  CUtensorMap k, q;  // q: [token][query head][D], boxes of N / G tokens x G heads x 64
};
struct WtBars {
  uint64_t *k_full, *k_empty, *q_full, *q_empty, *s_full, *s_empty;
  volatile int *stop;
};
__device__ __forceinline__ bool wait_all(const WtBars &B, uint64_t *bar, uint32_t parity) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = !*B.stop && mbar_wait(bar, parity);
  if (!ok) *B.stop = 1;
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A tile of 128 slots of request b and the rows (of one KV head: token * G + head) that see some of it.
struct SlotTile {
  Request rq;
  int b, j0, j1;       // first and last slot
  int base, used;
  int r_hi, t0, nt;    // row tiles t0 .. t0 + nt - 1; rows from r_hi on do not count
};
// The first row that does not see slot j any more for the window.
__device__ __forceinline__ int row_behind(const PagedArgs &a, const SlotTile &t, int j) {
  const int64_t i = static_cast<int64_t>(j) + a.window - t.base;
  return static_cast<int>(i < 0 ? 0 : i < t.used ? i : t.used) * a.group;
}
__device__ __forceinline__ int rows_used(const PagedWeightsArgs &A, const Request &rq, int b) {
  return A.rows_used ? max(0, min(__ldg(A.rows_used + b), rq.rows)) : rq.rows;
}
// The request's tiles that are gone through: without a window all of them, else the sinks' and those from
// the first row's window to the last row's slot; the slots between and behind them are shared out among those.
struct TileList {
  int sinks, first, count;
  __device__ int at(int t) const { return t < sinks ? t : first + t - sinks; }
};
__device__ __forceinline__ TileList tile_list(const PagedWeightsArgs &A, const Request &rq, int b) {
  const PagedArgs &a = A.p;
  TileList t = {0, 0, (rq.n + kTileSlots - 1) / kTileSlots};
  if (a.window == 0) return t;
  const int base = rq.n - rq.rows, last = base + rows_used(A, rq, b) - 1;  // the last row's slot
  if (last < max(0, base)) return t;  // no row that sees any
  const int first = window_first(a, max(0, base));
  t.first = first / kTileSlots;
  t.sinks = min((min(a.n_sink, first) + kTileSlots - 1) / kTileSlots, t.first);
  t.count = t.sinks + last / kTileSlots + 1 - t.first;
  return t;
}
// Request of list place `index`.
__device__ __forceinline__ int request_at(const int *before, int n, int index) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= index) lo = mid; else hi = mid;
  }
  return lo;
}
// Tile `index` of the list; NR rows make a row tile.
__device__ __forceinline__ SlotTile slot_tile(const PagedWeightsArgs &A, const int *before, int index, int NR) {
  const PagedArgs &a = A.p;
  SlotTile t;
  t.b = request_at(before, a.n_requests, index);
  t.rq = request_of(a, t.b);
  t.j0 = tile_list(A, t.rq, t.b).at(index - before[t.b]) * kTileSlots;
  t.j1 = min(t.j0 + kTileSlots, t.rq.n) - 1;
  t.base = t.rq.n - t.rq.rows;
  t.used = rows_used(A, t.rq, t.b);
  const int r_lo = max(0, t.j0 - t.base) * a.group;
  t.r_hi = a.window > 0 && t.j0 >= a.n_sink ? row_behind(a, t, t.j1) : t.used * a.group;
  t.t0 = r_lo / NR;
  t.nt = r_lo < t.r_hi ? (t.r_hi + NR - 1) / NR - t.t0 : 0;
  return t;
}
// before[b] = sum of count(0) .. count(b - 1); returns the sum of all.  All threads.
template <typename F> __device__ __forceinline__ int sum_up(const PagedArgs &a, int *before, int *warp_total, F count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = 0;
  for (int b0 = 0; b0 < a.n_requests; b0 += kThreads) {
    const int b = b0 + tid;
    int x = b < a.n_requests ? count(b) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_total[warp] = x;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) x += all;
      all += warp_total[w];
    }
    if (b < a.n_requests) before[b + 1] = n + x;
    n += all;
    __syncthreads();
  }
  if (tid == 0) before[0] = 0;
  __syncthreads();
  return n;
}

// The `place`th tile's part of the request's slots that no row sees: their scores only decay.  Thread wt of half
// `half` takes one slot of every other tile of them.
__device__ __forceinline__ void unseen_slots(const PagedWeightsArgs &A, const Request &rq, int b, int place, int half, int wt) {
  const TileList l = tile_list(A, rq, b);
  const int behind = l.first + l.count - l.sinks;  // first tile behind the seen ones
  const int gap = l.first - l.sinks, all = gap + (rq.n + kTileSlots - 1) / kTileSlots - behind;
  const int x1 = static_cast<int>(static_cast<int64_t>(all) * (place + 1) / l.count);
  for (int x0 = static_cast<int>(static_cast<int64_t>(all) * place / l.count) + half; x0 < x1; x0 += 8) {
    float v[4];
    int64_t at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = x0 + 2 * k, j = (x < gap ? l.sinks + x : behind + x - gap) * kTileSlots + wt;
      at[k] = x < x1 && j < rq.n ? b * A.score_stride + j : -1;
      v[k] = at[k] >= 0 && A.score_in ? A.decay * A.score_in[at[k]] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at[k] >= 0) A.score_out[at[k]] = v[k];
  }
}

template <typename T, int D, int N>
__global__ void __launch_bounds__(kThreads, 2) paged_weights_many(const __grid_constant__ PagedWeightsArgs A,
                                                                  const __grid_constant__ WeightMaps M, int box, int blocks) {
  using C = Wt<D, N>;
  constexpr int ATOMS = D / 64;
  constexpr uint32_t KS = C::kKSlots, QS = C::kQSlots;
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const PagedArgs &a = A.p;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x % blocks, cluster = blockIdx.x / blocks, clusters = gridDim.x / blocks;
  const int G = a.group, hq = a.n_kv_heads * G, tokens = N / G, NR = tokens * G;  // of a row tile
  const int heads = (a.n_kv_heads - rank + blocks - 1) / blocks;  // KV heads rank, rank + blocks, ...
  float *sums = reinterpret_cast<float *>(sm + C::kOffSum);
  int *before = reinterpret_cast<int *>(sm + C::kOffList);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  WtBars B;
  B.k_full = bars;
  B.k_empty = bars + KS;
  B.q_full = bars + 2 * KS;
  B.q_empty = B.q_full + QS;
  B.s_full = B.q_full + 2 * QS;
  B.s_empty = B.s_full + 2;
  uint64_t *drain = B.s_full + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  int *stop = reinterpret_cast<int *>(tmem_slot + 1);
  int *warp_total = stop + 1;  // [10]
  static_assert((2 * KS + 2 * QS + 5) * 8 + 8 + 40 <= 256, "barriers");
  B.stop = stop;
  if (tid == 0) {
    for (uint32_t i = 0; i < KS; ++i) {
      mbar_init(&B.k_full[i], 1);
      mbar_init(&B.k_empty[i], 1);
    }
    for (uint32_t i = 0; i < QS; ++i) {
      mbar_init(&B.q_full[i], 1);
      mbar_init(&B.q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.s_empty[i], 128);
    }
    mbar_init(drain, 1);
    *stop = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 8) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  const int n_tiles = sum_up(a, before, warp_total, [&](int b) {
    return a.window > 0 ? tile_list(A, request_of(a, b), b).count : (request_len(a, b) + kTileSlots - 1) / kTileSlots;
  });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // behind the allocation: a dependent kernel must not take the TMEM first and wait for this one
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 9) {  // loads
    const int n_boxes = kTileSlots / box * ATOMS;
    const bool mine = lane < n_boxes;
    const int bx = lane / ATOMS * box;
    uint32_t q = 0, k = 0;
    bool ok = true;
    for (int index = cluster; index < n_tiles; index += clusters) {
      const SlotTile t = slot_tile(A, before, index, NR);
      if (t.nt == 0) continue;
      const int j = t.j0 + bx;
      // beyond the pool (zeros): boxes of which no row that counts sees a slot
      int page = a.n_pages;
      if (mine && any_seen(a, j, box, window_first(a, max(0, t.base)), t.base + t.used - 1)) {
        page = __ldg(a.page_table + static_cast<int64_t>(t.b) * a.table_width + j / a.page_size);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
          page = a.n_pages;
          atomicOr(&g_error_word, DEVERR_BAD_INDEX);
        }
      }
      const int in_page = j % a.page_size;
      for (int x = 0; x < heads && ok; ++x, ++k) {
        const int h = rank + x * blocks;
        const uint32_t ks = k % KS;
        ok = k < KS || wait_all(B, &B.k_empty[ks], ((k / KS) - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&B.k_full[ks], C::kK);
        __syncwarp();
        if (mine)
          tma_load_4d(smem_u32(sm) + ks * C::kK + (lane % ATOMS) * kAtom + bx * 128, &M.k, &B.k_full[ks], (lane % ATOMS) * 64, in_page,
                      h, page);
        for (int r = 0; r < t.nt && ok; ++r, ++q) {
          const uint32_t slot = q % QS;
          ok = q < QS || wait_all(B, &B.q_empty[slot], ((q / QS) - 1) & 1);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&B.q_full[slot], NR * 128 * ATOMS);
          __syncwarp();
          if (lane < ATOMS)
            tma_load_3d(smem_u32(sm) + C::kOffQ + slot * C::kQ + lane * C::kQAtom, &M.q, &B.q_full[slot], lane * 64, h * G,
                        t.rq.row0 + (t.t0 + r) * tokens);
        }
      }
      __syncwarp();
      if (blocks > 1) cluster_sync();
    }
    // nothing is in flight when the block ends, after a wait that gave up either
    for (uint32_t i = k < KS ? 0 : k - KS; i < k; ++i) mbar_wait(&B.k_full[i % KS], (i / KS) & 1);
    for (uint32_t i = q < QS ? 0 : q - QS; i < q; ++i) mbar_wait(&B.q_full[i % QS], (i / QS) & 1);
  } else if (warp == 8) {  // products
    const uint32_t lead = elect_lead(), idesc = umma_idesc(ab_format<T>(), 128, N);
    const uint64_t k0 = umma_desc_sw128(smem_u32(sm)), q0 = umma_desc_sw128(smem_u32(sm) + C::kOffQ);
    uint32_t q = 0, k = 0;
    bool ok = true;
    for (int index = cluster; index < n_tiles; index += clusters) {
      const SlotTile t = slot_tile(A, before, index, NR);
      if (t.nt == 0) continue;
      for (int x = 0; x < heads && ok; ++x, ++k) {
        ok = wait_all(B, &B.k_full[k % KS], (k / KS) & 1);
        const uint64_t kd = k0 + (k % KS) * (C::kK >> 4);
        for (int r = 0; r < t.nt && ok; ++r, ++q) {
          const uint32_t slot = q % QS, half = q & 1;
          ok = wait_all(B, &B.q_full[slot], (q / QS) & 1) && (q < 2 || wait_all(B, &B.s_empty[half], ((q / 2) - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = q0 + slot * (C::kQ >> 4);
          mma_ss<false>(lead, tmem + half * N, kd, qd, idesc);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk)
            mma_ss<true>(lead, tmem + half * N, kd + (((kk >> 2) * kAtom + (kk & 3) * 32) >> 4),
                         qd + (((kk >> 2) * C::kQAtom + (kk & 3) * 32) >> 4), idesc);
          commit(lead, &B.s_full[half]);
          commit(lead, &B.q_empty[slot]);
        }
        if (ok) commit(lead, &B.k_empty[k % KS]);
      }
      __syncwarp();
      if (blocks > 1) cluster_sync();
    }
    commit(lead, drain);  // nothing is in flight when the TMEM is freed
    mbar_wait(drain, 0);
  } else {  // sums
    constexpr int CW = N < 32 ? N : 32;  // columns taken at a time
    const int half = warp >> 2, wt = tid & 127;
    const uint32_t ts = tmem + (static_cast<uint32_t>(wt & ~31) << 16) + half * N;
    float *lse_s = reinterpret_cast<float *>(sm + C::kOffLse) + half * 2 * N;
    uint32_t q = 0, turn = 0, n_s = 0;  // row tiles so far, sums' buffer, this half's row tiles
    bool ok = true;                     // false once a wait gave up: what follows only keeps the barriers
    for (int index = cluster; index < n_tiles; index += clusters) {
      const SlotTile t = slot_tile(A, before, index, NR);
      const int j = t.j0 + wt;
      float sum = 0.f;
      if (a.window > 0 && rank == 0) unseen_slots(A, t.rq, t.b, index - before[t.b], half, wt);  // while the keys come
      if (t.nt > 0) {
        // rows that see this thread's slot, and those that see all of the tile's
        const int lo = max(0, j - t.base) * G, hi = a.window > 0 && j >= a.n_sink ? row_behind(a, t, j) : t.used * G;
        const int all_lo = max(0, t.j1 - t.base) * G;
        const int all_hi = a.window > 0 && t.j1 >= a.n_sink ? row_behind(a, t, t.j0) : t.used * G;
        const float *lse = A.lse + static_cast<int64_t>(t.rq.row0) * hq;
        auto column = [&](int x, int r) {  // -log2(e) lse of this thread's column of row tile r, KV head number x
          const int row = (t.t0 + r) * NR + wt, i = row / static_cast<uint32_t>(G), e = row - i * G;
          return wt < NR && x < heads && row < t.r_hi ? __ldg(lse + static_cast<int64_t>(i) * hq + (rank + x * blocks) * G + e) * (-1.f / kLn2)
                                                     : -INFINITY;
        };
        uint64_t acc[2] = {0, 0};
        const int total = heads * t.nt;
        const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
        int u = (half ^ q) & 1;  // the tile's row tiles of this half: u, u + 2, ...
        int x = u / t.nt, r = u - x * t.nt;
        float next = column(x, r);
        for (; u < total; u += 2) {
          float *l_s = lse_s + (n_s & 1) * N;
          if (wt < N) l_s[wt] = next;
          named_bar(1 + half, 128);
          const int r0 = (t.t0 + r) * NR;
          for (r += 2; r >= t.nt && x < heads; r -= t.nt) ++x;
          next = column(x, r);
          ok = ok && wait_all(B, &B.s_full[half], n_s & 1);
          ++n_s;
          tc_fence_after();
          const bool edge = r0 < all_lo || r0 + N > all_hi || NR < N;  // columns from NR on are no rows
          const int end = min(hi, r0 + NR);
#pragma unroll 1
          for (int k = 0; k < N; k += CW) {
            uint32_t w[CW];
            if constexpr (CW == 32) {
              tmem_ld32_nowait(ts + k, w);
              tmem_ld_wait();
              tmem_values(w);
            } else {
              float f[16];
              tmem_ld16(ts, f);
#pragma unroll
              for (int c = 0; c < 16; ++c) w[c] = __float_as_uint(f[c]);
            }
            if (!edge) {
#pragma unroll
              for (int c = 0; c < CW; c += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(l_s + k + c);
                const float2 y0 = unpair(fma2(pair_bits(w[c], w[c + 1]), scale2, pair(l.x, l.y)));
                const float2 y1 = unpair(fma2(pair_bits(w[c + 2], w[c + 3]), scale2, pair(l.z, l.w)));
                acc[0] = add2(acc[0], pair(exp2_fast(y0.x), exp2_fast(y0.y)));
                acc[1] = add2(acc[1], pair(exp2_fast(y1.x), exp2_fast(y1.y)));
              }
            } else {  // a hidden column adds nothing, whatever its row and lse hold
              const uint32_t bits = seen_bits(end - 1 - r0 - k, lo - r0 - k, 0);
#pragma unroll
              for (int c = 0; c < CW; ++c) {
                const float y = exp2_fast(fmaf(__uint_as_float(w[c]), a.scale_log2, l_s[k + c]));
                if (bits & (1u << c)) sum += y;
              }
            }
          }
          tc_fence_before();
          mbar_arrive(&B.s_empty[half]);
        }
        q += total;
        const float2 y = unpair(add2(acc[0], acc[1]));
        sum += y.x + y.y;
        // both halves' and all blocks' sums; two sets, so that a tile's are read before the next but one's come
        float *set = sums + (turn & 1) * 256;
        ++turn;
        set[half * 128 + wt] = sum;
        if (blocks > 1) cluster_sync(); else named_bar(3, 256);
        sum = 0.f;
        if (half == 0 && rank == 0)
          for (int p = 0; p < blocks; ++p) {
            if (blocks == 1) {
              sum = set[wt] + set[128 + wt];
            } else {
              const uint32_t at = cluster_map(smem_u32(set + wt), p);
              sum += ld_cluster_f32(at) + ld_cluster_f32(at + 512);
            }
          }
      }
      if (half == 0 && rank == 0 && j < t.rq.n) {
        const int64_t at = t.b * A.score_stride + j;
        A.score_out[at] = (A.score_in ? A.decay * A.score_in[at] : 0.f) + sum;
      }
    }
  }
  tc_fence_before();
  if (blocks > 1) cluster_sync(); else __syncthreads();  // every block's sums are read
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, C::kCols);
}

template <typename T, int D, int N> cudaError_t launch(const PagedWeightsArgs &A, const WeightMaps &M, int box, cudaStream_t s) {
  const PagedArgs &a = A.p;
  const cudaError_t e = cudaFuncSetAttribute(paged_weights_many<T, D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Wt<D, N>::kSmem);
  if (e != cudaSuccess) return e;
  // Blocks that share the KV heads of a tile: as many as make the longest block's work -- its tiles times
  // their heads, and about one more for each, three where blocks meet -- the shortest (one request of
  // 16 384 slots, 129 tiles, 8 heads: two blocks 9.3 us, four 15.5 us).
  const int64_t most = (a.max_len + kTileSlots - 1) / kTileSlots * static_cast<int64_t>(a.n_requests);
  const int64_t tiles = (visible_slots(a) / kTileSlots + 1) * a.n_requests;
  int blocks = 1;
  int64_t best = INT64_MAX;
  for (int x = 1; x <= kMaxBlocks && x <= a.n_kv_heads; x *= 2) {
    const int64_t at_once = 2 * num_sms() / x, work = (tiles + at_once - 1) / at_once * ((a.n_kv_heads + x - 1) / x + (x > 1 ? 3 : 1));
    if (work < best) {
      best = work;
      blocks = x;
    }
  }
  const int64_t room = 2 * num_sms() / blocks, clusters = most < room ? most : room;
  return launch_pdl_cluster(paged_weights_many<T, D, N>, dim3(static_cast<unsigned>(clusters * blocks)), dim3(kThreads), Wt<D, N>::kSmem,
                            s, blocks, A, M, box, blocks);
}
template <typename T, int D> cudaError_t launch_rows(const PagedWeightsArgs &A, const WeightMaps &M, int box, int n, cudaStream_t s) {
  return n == 16 ? launch<T, D, 16>(A, M, box, s) : n == 64 ? launch<T, D, 64>(A, M, box, s) : launch<T, D, 128>(A, M, box, s);
}
int row_tile(const PagedArgs &a) {
  const int rows = a.max_rows * a.group;
  return rows <= 16 ? 16 : rows <= 64 ? 64 : 128;
}

}  // namespace

// Whether the kernel above takes the call: pages must make whole boxes.
bool weights_many_takes(const PagedArgs &a) { return a.max_rows > 0 && box_rows(a.page_size) > 0; }

std::string launch_weights_many(const PagedWeightsArgs &A, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  const bool bf16 = dtype == BD_BF16;
  const int box = box_rows(a.page_size), n = row_tile(a);
  WeightMaps M;
  const int hq = a.n_kv_heads * a.group;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.head_dim), static_cast<cuuint64_t>(hq), static_cast<cuuint64_t>(a.n_rows)};
  const int64_t stride[2] = {a.head_dim, a.q_stride};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(n / a.group)};
  if (!pool_map(&M.k, a, a.k, bf16, box) || !tiled_map(&M.q, a.q, bf16, 3, dims, stride, boxes))
    return "paged weights: cuTensorMapEncodeTiled failed";
  cudaError_t e;
  if (bf16)
    e = a.head_dim == 128 ? launch_rows<__nv_bfloat16, 128>(A, M, box, n, s) : launch_rows<__nv_bfloat16, 64>(A, M, box, n, s);
  else
    e = a.head_dim == 128 ? launch_rows<__half, 128>(A, M, box, n, s) : launch_rows<__half, 64>(A, M, box, n, s);
  return e == cudaSuccess ? std::string() : std::string("paged weights: ") + cudaGetErrorString(e);
}

}  // namespace bd
