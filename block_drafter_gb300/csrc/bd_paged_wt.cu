// Accumulated attention weights of many rows (bd_paged_weights) on the tensor cores.
//
// S^T = K Q^T with the slots on the MMA's M side: a thread owns one slot -- one TMEM lane -- and adds up
// its weights 2^(scale log2(e) s - log2(e) lse) over the columns, which are the rows, in a register.  So
// nothing crosses lanes, and a slot that holds anything at all touches its own lane only.  A block takes
// 128 slots and one KV head (or every kth) of a request and passes over the rows that see them, 128 at a
// time; a cluster's blocks share the KV heads and add their sums through distributed shared memory, in
// rank order.  Bound by the exponentials and the tensor cores alike (a 128 x 128 tile: 512 cycles each on
// an SM), for few rows by the chain load - product - sum.
//   warps 0-3, 4-7  take the row tiles in turn, each from its half of TMEM (128 columns)
//   warp 8          issues the MMAs;  warp 9  brings K and Q by TMA
// Two blocks on an SM hide each other's start.
#include "bd_paged_tc.cuh"

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged_wt)

namespace {

constexpr int kThreads = 320;
constexpr int kQSlots = 2;     // row tiles in shared memory
constexpr int kMaxBlocks = 8;  // of a cluster

template <int D> struct Wt {
  static constexpr uint32_t kTile = (D / 64) * kAtom;
  static constexpr uint32_t kOffQ = kTile;
  static constexpr uint32_t kOffLse = kOffQ + kQSlots * kTile;  // [2 halves][2 turns][128] floats
  static constexpr uint32_t kOffSum = kOffLse + 2048;           // [2][128]
  static constexpr uint32_t kOffBar = kOffSum + 1024;
  static constexpr size_t kSmem = 1024 + kOffBar + 128;
};
struct WeightMaps {
  CUtensorMap k, q;  // q: [token][query head][D], boxes of 128 / G tokens x G heads x 64
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) paged_weights_many(const __grid_constant__ PagedWeightsArgs A,
                                                                  const __grid_constant__ WeightMaps M, int box) {
  using C = Wt<D>;
  constexpr int ATOMS = D / 64;
  extern __shared__ uint8_t sm_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const PagedArgs &a = A.p;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x, blocks = gridDim.x, b = blockIdx.z, j0 = blockIdx.y * kTileSlots;
  pdl_wait();
  const Request rq = request_of(a, b);
  if (j0 >= rq.n) return;  // the whole cluster
  const int used = A.rows_used ? max(0, min(A.rows_used[b], rq.rows)) : rq.rows;
  const int G = a.group, hq = a.n_kv_heads * G, base = rq.n - rq.rows, j1 = min(j0 + kTileSlots, rq.n) - 1;
  // rows that see some slot of the tile: r_lo .. r_hi - 1 (rows of one KV head: token * G + head)
  auto behind = [&](int j) {  // the first row that does not see slot j any more for its window
    const int64_t i = static_cast<int64_t>(j) + a.window - base;
    return static_cast<int>(i < 0 ? 0 : i < used ? i : used) * G;
  };
  const int r_lo = max(0, j0 - base) * G, r_hi = a.window > 0 && j0 >= a.n_sink ? behind(j1) : used * G;
  const int t0 = r_lo / 128, t1 = r_lo < r_hi ? (r_hi + 127) / 128 : t0;  // row tiles
  float *sums = reinterpret_cast<float *>(sm + C::kOffSum);
  if (t0 == t1) {  // nobody sees them
    if (rank == 0 && tid < 128 && j0 + tid < rq.n) {
      const int64_t at = b * A.score_stride + j0 + tid;
      A.score_out[at] = A.score_in ? A.decay * A.score_in[at] : 0.f;
    }
    return;
  }
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  WtBars B;
  B.k_full = bars;
  B.k_empty = bars + 1;
  B.q_full = bars + 2;
  B.q_empty = bars + 2 + kQSlots;
  B.s_full = bars + 2 + 2 * kQSlots;
  B.s_empty = B.s_full + 2;
  uint64_t *drain = B.s_full + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  int *stop = reinterpret_cast<int *>(tmem_slot + 1);
  B.stop = stop;
  if (tid == 0) {
    mbar_init(B.k_full, 1);
    mbar_init(B.k_empty, 1);
    for (int i = 0; i < kQSlots; ++i) {
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
  if (warp == 8) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  if (tid < 256) sums[tid] = 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // behind the allocation: a dependent kernel must not take the TMEM first and wait for this one
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int heads = (a.n_kv_heads - rank + blocks - 1) / blocks, nt = t1 - t0;  // KV heads rank, rank + blocks, ...

  if (warp == 9) {  // loads
    const int n_boxes = kTileSlots / box * ATOMS;
    const bool mine = lane < n_boxes;
    const int bx = lane / ATOMS * box, j = j0 + bx;
    int page = a.n_pages;  // beyond the pool: zeros
    if (mine && j < rq.n) {
      page = __ldg(a.page_table + static_cast<int64_t>(b) * a.table_width + j / a.page_size);
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
        page = a.n_pages;
        atomicOr(&g_error_word, DEVERR_BAD_INDEX);
      }
    }
    uint32_t q = 0;
    bool ok = true;
    for (int x = 0; x < heads && ok; ++x) {
      const int h = rank + x * blocks;
      if (x > 0) ok = wait_all(B, B.k_empty, (x - 1) & 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(B.k_full, C::kTile);
      __syncwarp();
      if (mine)
        tma_load_4d(smem_u32(sm) + (lane % ATOMS) * kAtom + bx * 128, &M.k, B.k_full, (lane % ATOMS) * 64, j % a.page_size, h, page);
      for (int t = t0; t < t1; ++t, ++q) {
        const uint32_t slot = q % kQSlots;
        if (q >= kQSlots && !wait_all(B, &B.q_empty[slot], ((q / kQSlots) - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&B.q_full[slot], C::kTile);
        __syncwarp();
        if (lane < ATOMS)
          tma_load_3d(smem_u32(sm) + C::kOffQ + slot * C::kTile + lane * kAtom, &M.q, &B.q_full[slot], lane * 64, h * G,
                      rq.row0 + t * 128 / G);
      }
    }
  } else if (warp == 8) {  // products
    const uint32_t lead = elect_lead(), idesc = umma_idesc(ab_format<T>(), 128, 128);
    const uint64_t k0 = umma_desc_sw128(smem_u32(sm)), q0 = umma_desc_sw128(smem_u32(sm) + C::kOffQ);
    uint32_t q = 0;
    bool ok = true;
    for (int x = 0; x < heads && ok; ++x) {
      ok = wait_all(B, B.k_full, x & 1);
      for (int t = 0; t < nt && ok; ++t, ++q) {
        const uint32_t slot = q % kQSlots, half = q & 1;
        ok = wait_all(B, &B.q_full[slot], (q / kQSlots) & 1) && (q < 2 || wait_all(B, &B.s_empty[half], ((q / 2) - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = q0 + slot * (C::kTile >> 4);
        mma_ss<false>(lead, tmem + half * 128, k0, qd, idesc);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4;
          mma_ss<true>(lead, tmem + half * 128, k0 + off, qd + off, idesc);
        }
        commit(lead, &B.s_full[half]);
        commit(lead, &B.q_empty[slot]);
      }
      if (ok) commit(lead, B.k_empty);
    }
    commit(lead, drain);  // nothing is in flight when the TMEM is freed
    mbar_wait(drain, 0);
  } else {  // sums
    const int half = warp >> 2, wt = tid & 127, j = j0 + wt;
    const uint32_t ts = tmem + (static_cast<uint32_t>(wt & ~31) << 16) + half * 128;
    float *lse_s = reinterpret_cast<float *>(sm + C::kOffLse) + half * 256;
    // rows that see this thread's slot
    const int lo = max(0, j - base) * G, hi = a.window > 0 && j >= a.n_sink ? behind(j) : used * G;
    // rows that see all of the tile's slots
    const int all_lo = max(0, j1 - base) * G, all_hi = a.window > 0 && j1 >= a.n_sink ? behind(j0) : used * G;
    const float *lse = A.lse + static_cast<int64_t>(rq.row0) * hq;
    uint64_t acc[2] = {0, 0};
    const int total = heads * nt;
    int x = 0, t = half;  // head and row tile of q
    bool ok = true;       // false once a wait gave up: what follows only keeps the barrier
    while (t >= nt && x < heads) t -= nt, ++x;
    for (int q = half; q < total; q += 2) {
      float *l_s = lse_s + ((q >> 1) & 1) * 128;
      const int r0 = (t0 + t) * 128, h = rank + x * blocks;
      {
        const int r = r0 + wt, i = r / static_cast<uint32_t>(G), e = r - i * G;
        l_s[wt] = r < r_hi ? __ldg(lse + static_cast<int64_t>(i) * hq + h * G + e) * (-1.f / kLn2) : -INFINITY;
      }
      named_bar(1 + half, 128);
      ok = ok && wait_all(B, &B.s_full[half], (q >> 1) & 1);
      tc_fence_after();
      const bool edge = r0 < all_lo || r0 + 128 > all_hi;
      const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t w[32];
        tmem_ld32_nowait(ts + 32 * k, w);
        tmem_ld_wait();
        tmem_values(w);
        const int c0 = r0 + 32 * k;
        const uint32_t bits = edge ? seen_bits(hi - 1 - c0, lo - c0, 0) : ~0u;  // columns lo .. hi - 1 count
        if (!edge) {
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 l = *reinterpret_cast<const float4 *>(l_s + 32 * k + c);
            const float2 y0 = unpair(fma2(pair_bits(w[c], w[c + 1]), scale2, pair(l.x, l.y)));
            const float2 y1 = unpair(fma2(pair_bits(w[c + 2], w[c + 3]), scale2, pair(l.z, l.w)));
            acc[0] = add2(acc[0], pair(exp2_fast(y0.x), exp2_fast(y0.y)));
            acc[1] = add2(acc[1], pair(exp2_fast(y1.x), exp2_fast(y1.y)));
          }
        } else {
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < 32; ++c) {  // a hidden column adds nothing, whatever its row and lse hold
            const float y = exp2_fast(fmaf(__uint_as_float(w[c]), a.scale_log2, l_s[32 * k + c]));
            if (bits & (1u << c)) sum += y;
          }
          acc[0] = add2(acc[0], pair(sum, 0.f));
        }
      }
      tc_fence_before();
      mbar_arrive(&B.s_empty[half]);
      for (t += 2; t >= nt && x < heads; t -= nt) ++x;
    }
    const float2 s = unpair(add2(acc[0], acc[1]));
    sums[half * 128 + wt] = s.x + s.y;
  }
  tc_fence_before();
  if (blocks > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  if (rank == 0 && tid < 128 && j0 + tid < rq.n) {
    float s = 0.f;
    if (blocks == 1) {
      s = sums[tid] + sums[128 + tid];
    } else {
      for (int r = 0; r < blocks; ++r) {
        const uint32_t at = cluster_map(smem_u32(sums + tid), r);
        s += ld_cluster_f32(at) + ld_cluster_f32(at + 512);
      }
    }
    const int64_t at = b * A.score_stride + j0 + tid;
    A.score_out[at] = (A.score_in ? A.decay * A.score_in[at] : 0.f) + s;
  }
  if (blocks > 1) cluster_sync();  // the sums are read
  if (warp == 8) tmem_dealloc(tmem, 256);
}

template <typename T, int D> cudaError_t launch(const PagedWeightsArgs &A, const WeightMaps &M, int box, cudaStream_t s) {
  const PagedArgs &a = A.p;
  const cudaError_t e = cudaFuncSetAttribute(paged_weights_many<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Wt<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int blocks = a.n_kv_heads < kMaxBlocks ? a.n_kv_heads : kMaxBlocks;
  return launch_pdl_cluster(paged_weights_many<T, D>, dim3(blocks, (a.max_len + kTileSlots - 1) / kTileSlots, a.n_requests),
                            dim3(kThreads), Wt<D>::kSmem, s, blocks, A, M, box);
}

}  // namespace

// Whether the kernel above takes the call: pages and head groups must make whole boxes, and the grid hold
// the tiles.
bool weights_many_takes(const PagedArgs &a) {
  return box_rows(a.page_size) > 0 && 128 % a.group == 0 && (a.max_len + kTileSlots - 1) / kTileSlots <= 65535;
}

std::string launch_weights_many(const PagedWeightsArgs &A, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  const bool bf16 = dtype == BD_BF16;
  const int box = box_rows(a.page_size);
  WeightMaps M;
  const int hq = a.n_kv_heads * a.group;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.head_dim), static_cast<cuuint64_t>(hq), static_cast<cuuint64_t>(a.n_rows)};
  const int64_t stride[2] = {a.head_dim, a.q_stride};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(a.group), static_cast<cuuint32_t>(128 / a.group)};
  if (!pool_map(&M.k, a, a.k, bf16, box) || !tiled_map(&M.q, a.q, bf16, 3, dims, stride, boxes))
    return "paged weights: cuTensorMapEncodeTiled failed";
  cudaError_t e;
  if (bf16)
    e = a.head_dim == 128 ? launch<__nv_bfloat16, 128>(A, M, box, s) : launch<__nv_bfloat16, 64>(A, M, box, s);
  else
    e = a.head_dim == 128 ? launch<__half, 128>(A, M, box, s) : launch<__half, 64>(A, M, box, s);
  return e == cudaSuccess ? std::string() : std::string("paged weights: ") + cudaGetErrorString(e);
}

}  // namespace bd
