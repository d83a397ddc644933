// Paged K/V cache: the entry points' checks, and the kernels of the append, the accumulated
// attention weights and the eviction.
#include "bd_paged_attn.cuh"

#include <climits>
#include <cmath>

namespace bd {

BD_DEFINE_ERROR_TAKER(take_error_word_paged)

static std::atomic<bool> paged_used{false};  // some call of this file has launched, or been captured
unsigned take_error_words_paged() {
  if (!paged_used.load(std::memory_order_acquire)) return 0;
  return take_error_word_paged() | take_error_word_paged_attn() | take_error_word_paged_tc() | take_error_word_paged_wt();
}

// ------------------------------------------------------------------ append
// Copies each row's keys and values into its slot.  A block takes rows_per_cta consecutive rows; the first
// kAppendEach 16-byte pieces of every thread are on their way while it finds the rows' requests -- every
// thread tests some of the requests' row ranges against the block's -- and slots.  Bound by the bytes
// (23 700 rows of 8 heads 33.4 us, 5.8 TB/s read and written), of few rows by the launch (2.5 us).
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 32;
constexpr int kAppendEach = 4;

struct PagedAppendArgs {
  PagedArgs p;
  const void *k_new, *v_new;
  int64_t k_stride, v_stride;
  int rows_per_cta;
};

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ PagedAppendArgs A) {
  const PagedArgs &a = A.p;
  __shared__ int64_t off[kAppendRows];  // element offset of the row's slot, -1: not stored
  __shared__ int2 place[kAppendRows];   // the row's request and slot (negative: none)
  const int r0 = blockIdx.x * A.rows_per_cta, r1 = min(a.n_rows, r0 + A.rows_per_cta);
  const uint32_t per_head = a.head_dim / 8, per_side = a.n_kv_heads * per_head, per_row = 2 * per_side;
  const int pieces = (r1 - r0) * per_row;
  if (threadIdx.x < kAppendRows) place[threadIdx.x] = make_int2(0, -1);
  pdl_wait();
  pdl_trigger();
  uint4 v[kAppendEach];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < kAppendEach; ++u) {
      const uint32_t c = c0 + u * kAppendThreads, r = c / per_row, x = c - r * per_row;
      if (c >= pieces) continue;
      const void *row = x < per_side ? static_cast<const uint16_t *>(A.k_new) + (r0 + r) * A.k_stride + x * 8
                                     : static_cast<const uint16_t *>(A.v_new) + (r0 + r) * A.v_stride + (x - per_side) * 8;
      v[u] = __ldcs(static_cast<const uint4 *>(row));
    }
  };
  load(threadIdx.x);
  __syncthreads();
  for (int b = threadIdx.x; b < a.n_requests; b += kAppendThreads) {
    const int s = a.row_start[b], e = a.row_start[b + 1], n = request_len(a, b);
    if (s < 0 || e < s || e > a.n_rows || e - s > a.max_rows) {
      atomicOr(&g_error_word, DEVERR_BAD_INDEX);
      continue;
    }
    for (int r = max(s, r0); r < min(e, r1); ++r) place[r - r0] = make_int2(b, n - (e - r));
  }
  __syncthreads();
  if (threadIdx.x < kAppendRows) {
    const int2 p = place[threadIdx.x];
    off[threadIdx.x] = p.y < 0 ? -1 : slot_offset(a, a.page_table + static_cast<int64_t>(p.x) * a.table_width, p.y);
  }
  __syncthreads();
  for (int c0 = threadIdx.x; c0 < pieces; c0 += kAppendEach * kAppendThreads) {
    if (c0 != static_cast<int>(threadIdx.x)) load(c0);
#pragma unroll
    for (int u = 0; u < kAppendEach; ++u) {
      const uint32_t c = c0 + u * kAppendThreads, r = c / per_row, x = c - r * per_row;
      if (c >= pieces || off[r] < 0) continue;
      const uint32_t w = x < per_side ? x : x - per_side, h = w / per_head;
      uint16_t *to = static_cast<uint16_t *>(const_cast<void *>(x < per_side ? a.k : a.v));
      *reinterpret_cast<uint4 *>(to + off[r] + h * a.head_stride + (w - h * per_head) * 8) = v[u];
    }
  }
}

static std::string launch_append(PagedAppendArgs &A, cudaStream_t s) {
  // as many rows as its threads' first pieces cover, while two blocks an SM are left (22 000 rows of one head of
  // 128 in blocks of four 11.8 us, of thirty-two 6.3 us)
  const int pieces = 2 * A.p.n_kv_heads * A.p.head_dim / 8;
  A.rows_per_cta = 1;
  while (2 * A.rows_per_cta <= kAppendRows && 2 * A.rows_per_cta * pieces <= kAppendEach * kAppendThreads &&
         A.p.n_rows >= 4 * A.rows_per_cta * num_sms())
    A.rows_per_cta *= 2;
  const int grid = (A.p.n_rows + A.rows_per_cta - 1) / A.rows_per_cta;
  const cudaError_t e = launch_pdl(paged_append_kernel, dim3(grid), dim3(kAppendThreads), 0, s, A);
  return e == cudaSuccess ? std::string() : std::string("paged append: ") + cudaGetErrorString(e);
}

// ------------------------------------------------------------------ accumulated weights
// out[j] = decay in[j] + sum over rows i and heads of 2^(scale log2(e) k_j.q_i - log2(e) lse_i).
// For pages whose slots make no TMA boxes; others go to the persistent kernel (8 requests of 8192 slots, 16 rows
// of group 3: 29 us there, 79 us here).  A warp owns 16 slots of
// a request: their keys are the A operand of mma.sync m16n8k16 and stay in registers while the rows of
// the KV head pass by, 8 at a time, as B; so a slot's weights are summed in the registers of four lanes,
// without atomics, over all rows and heads of the warp.
// The order of the D products of a score is free, so both operands are taken as 16-byte pieces: lane l
// holds pieces l%4, l%4 + 4, ... of its rows, two MMA steps each.
constexpr int kWeightWarps = 8;

template <typename T> __device__ __forceinline__ void mma_kq(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_kq<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_kq<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile of 16 slots of a request, and which tokens (of slot base + i) it concerns.
struct WeightTile {
  Request rq;
  int b, j0, base;
  int last;          // slot of the last token that counts
  int i_lo, i_hi;    // tokens that see some of its slots
  int f_lo, f_hi;    // rows that see all of them, f_lo to f_hi - 1
  int64_t q0;        // this lane's row of the first row tile: element offset in q (KV head 0),
  int lse0, i0, e0;  //   offset in lse from the request's first row, token, head of the group
};
__device__ __forceinline__ WeightTile weight_tile(const PagedWeightsArgs &A, int b, int j0, int quad, int kq) {
  const PagedArgs &a = A.p;
  WeightTile t;
  t.rq = request_of(a, b);
  t.b = b;
  t.j0 = j0;
  t.base = t.rq.n - t.rq.rows;
  const int used = A.rows_used ? max(0, min(__ldg(A.rows_used + b), t.rq.rows)) : t.rq.rows;
  const int j1 = min(j0 + 15, t.rq.n - 1);
  t.last = t.base + used - 1;
  t.i_lo = max(0, j0 - t.base);
  t.f_lo = max(0, j1 - t.base);
  t.i_hi = t.f_hi = used;
  if (a.window > 0) {
    auto behind = [&](int j) {  // the first token that does not see slot j any more, 0 .. used
      const int64_t i = static_cast<int64_t>(j) + a.window - t.base;
      return static_cast<int>(i < 0 ? 0 : i < used ? i : used);
    };
    if (j0 >= a.n_sink) t.i_hi = behind(j1);
    if (j1 >= a.n_sink) t.f_hi = behind(j0);
  }
  if (t.f_hi == t.i_hi) t.f_hi = INT_MAX;  // rows behind the last count nothing anyway
  else t.f_hi *= a.group;
  t.f_lo *= a.group;
  const uint32_t r0 = t.i_lo * a.group / 8 * 8 + quad;
  t.i0 = r0 / static_cast<uint32_t>(a.group);
  t.e0 = r0 - t.i0 * a.group;
  t.q0 = (t.rq.row0 + t.i0) * a.q_stride + t.e0 * a.head_dim + kq * 8;
  t.lse0 = t.i0 * a.n_kv_heads * a.group + t.e0;
  return t;
}

// How a lane steps from a row tile to the next: 8 rows are di tokens and de heads on, or one token more
// and a group less.
struct RowStep {
  int di, de, dl, wrap_l;
  int64_t dq, wrap_q;
};

// Weights a tile's slots (quad, quad + 8) get from the rows of KV head h, its keys in kf: added to acc.
template <typename T, int D>
__device__ __forceinline__ void tile_weights(const PagedWeightsArgs &A, const WeightTile &w, const RowStep &rs, int h,
                                             const uint32_t (&kf)[D / 16][4], float (&acc)[2], int quad, int kq) {
  constexpr int P = D / 32;
  const PagedArgs &a = A.p;
  const int G = a.group;
  const int t0 = w.i_lo * G / 8, t1 = (w.i_hi * G + 7) / 8;  // row tiles of 8
  const T *q = static_cast<const T *>(a.q) + w.q0 + h * G * D;
  const float *lse = A.lse + static_cast<int64_t>(w.rq.row0) * a.n_kv_heads * G + w.lse0 + h * G;
  int i = w.i0, e = w.e0;
  uint4 qn[P];
  float ln = INFINITY;  // no weight behind the last row
#pragma unroll
  for (int c = 0; c < P; ++c) qn[c] = make_uint4(0, 0, 0, 0);
  auto fetch = [&]() {
    if (i < w.i_hi) {
      ln = __ldg(lse);
#pragma unroll
      for (int c = 0; c < P; ++c) qn[c] = __ldg(reinterpret_cast<const uint4 *>(q) + 4 * c);
    } else {
      ln = INFINITY;
    }
  };
  fetch();
#pragma unroll 2
  for (int t = t0; t < t1; ++t) {
    float c0[4] = {}, c1[4] = {};
#pragma unroll
    for (int c = 0; c < P; ++c) {
      mma_kq<T>(c0, kf[2 * c], qn[c].x, qn[c].y);
      mma_kq<T>(c1, kf[2 * c + 1], qn[c].z, qn[c].w);
    }
    const float l = ln * (1.f / kLn2);
    const int token = i;
    i += rs.di;
    e += rs.de;
    q += rs.dq;
    lse += rs.dl;
    if (e >= G) {
      e -= G;
      ++i;
      q += rs.wrap_q;
      lse += rs.wrap_l;
    }
    if (t + 1 < t1) fetch();
    // columns of this lane: rows 2 kq and 2 kq + 1 of the row tile
    const float l0 = __shfl_sync(0xffffffffu, l, 8 * kq), l1 = __shfl_sync(0xffffffffu, l, 8 * kq + 4);
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float lx = x & 1 ? l1 : l0;
      v[x] = lx == INFINITY ? 0.f : exp2_fast(fmaf(c0[x] + c1[x], a.scale_log2, -lx));
    }
    if (t * 8 < w.f_lo || t * 8 + 8 > w.f_hi) {
      const int p0 = w.base + __shfl_sync(0xffffffffu, token, 8 * kq), p1 = w.base + __shfl_sync(0xffffffffu, token, 8 * kq + 4);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int p = x & 1 ? p1 : p0, j = w.j0 + quad + (x & 2 ? 8 : 0);
        if (!(p >= 0 && j <= p && (j >= window_first(a, p) || j < a.n_sink))) v[x] = 0.f;
      }
    }
    acc[0] += v[0] + v[1];
    acc[1] += v[2] + v[3];
  }
}

// Blocks of the weights kernel: two on every SM.  Each of its teams of head_split warps takes every
// n_teams-th slot tile of the call's list (all requests' tiles in order); the tile's KV heads hs,
// hs + head_split, ... are warp hs's.  A warp's keys -- one KV head of one tile a stage -- come by cp.async
// into its own ring, kStages - 1 ahead across heads and tiles.
template <int D> struct Weights {
  static constexpr int kStage = 16 * 2 * D;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kSmem = kWeightWarps * kStages * kStage;
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWeightWarps, 2) paged_weights_kernel(const __grid_constant__ PagedWeightsArgs A, int head_split) {
  using W = Weights<D>;
  constexpr int CPR = D / 8, RPI = 32 / CPR, P = D / 32;
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ int tiles_before[BD_PAGED_MAX_REQUESTS + 1];
  __shared__ float part[2][kWeightWarps][16];
  __shared__ int warp_total[kWeightWarps];
  const PagedArgs &a = A.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = lane >> 2, kq = lane & 3;
  pdl_wait();
  pdl_trigger();
  {  // tiles of the requests before each
    int before = 0;
    for (int b0 = 0; b0 < a.n_requests; b0 += 32 * kWeightWarps) {
      const int b = b0 + tid;
      int x = b < a.n_requests ? (request_len(a, b) + 15) / 16 : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_total[warp] = x;
      __syncthreads();
      int all = 0;
      for (int w = 0; w < kWeightWarps; ++w) {
        if (w == warp) x += all;
        all += warp_total[w];
      }
      if (b < a.n_requests) tiles_before[b + 1] = before + x;
      before += all;
      __syncthreads();
    }
    if (tid == 0) tiles_before[0] = 0;
    __syncthreads();
  }
  const int n_tiles = tiles_before[a.n_requests];
  const int teams = kWeightWarps / head_split, n_teams = teams * gridDim.x;
  const int hs = warp / teams, heads = hs < a.n_kv_heads ? (a.n_kv_heads - hs + head_split - 1) / head_split : 0;
  const int first = blockIdx.x + (warp % teams) * gridDim.x;  // a block's teams lie far apart in the list
  auto tile_at = [&](int t) {
    int lo = 0, hi = a.n_requests;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tiles_before[mid] <= t) lo = mid; else hi = mid;
    }
    return weight_tile(A, lo, (t - tiles_before[lo]) * 16, quad, kq);
  };
  RowStep rs;
  rs.di = 8 / a.group;
  rs.de = 8 - rs.di * a.group;
  rs.dl = rs.di * a.n_kv_heads * a.group + rs.de;
  rs.wrap_l = (a.n_kv_heads - 1) * a.group;
  rs.dq = rs.di * a.q_stride + rs.de * D;
  rs.wrap_q = a.q_stride - a.group * D;
  const uint32_t mine = smem_u32(ring) + warp * W::kStages * W::kStage;
  // the copies run ahead of the products: their own place in the list
  int ct = first, ch = 0;
  int64_t off[16 / RPI];  // of the rows this lane copies, -1: none
  bool any = false;       // some row sees some of the tile
  auto open = [&]() {
    if (ct >= n_tiles) return;
    const WeightTile w = tile_at(ct);
    any = w.i_lo < w.i_hi && heads > 0;
    const int j = w.j0 + (lane & 15);
    const int64_t o = any && any_seen(a, j, 1, window_first(a, max(0, w.base)), w.last) ? slot_offset(a, a.page_table + static_cast<int64_t>(w.b) * a.table_width, j) : -1;
#pragma unroll
    for (int u = 0; u < 16 / RPI; ++u) {
      off[u] = __shfl_sync(0xffffffffu, o, u * RPI + lane / CPR);
      if (off[u] >= 0) off[u] += lane % CPR * 8;
    }
  };
  auto copy = [&](int stage) {  // one KV head of one tile
    while (ct < n_tiles && !any) {  // tiles nobody sees
      ct += n_teams;
      open();
    }
    if (ct < n_tiles) {
      const T *K = static_cast<const T *>(a.k) + (hs + ch * head_split) * a.head_stride;
      const uint32_t dst = mine + stage * W::kStage;
      const int c = lane % CPR;
#pragma unroll
      for (int u = 0; u < 16 / RPI; ++u) {
        const int r = u * RPI + lane / CPR;
        cp_async16(dst + r * 2 * D + ((c ^ (r & 7)) << 4), K + (off[u] < 0 ? 0 : off[u]), off[u] >= 0);
      }
      if (++ch == heads) {
        ch = 0;
        ct += n_teams;
        open();
      }
    }
    cp_async_commit();
  };
  open();
#pragma unroll
  for (int st = 0; st < W::kStages - 1; ++st) copy(st);
  int stage = 0, turn = 0;
  for (int t = first; t < n_tiles; t += n_teams) {
    const WeightTile w = tile_at(t);
    float acc[2] = {0.f, 0.f};  // slots j0 + quad, + 8
    if (w.i_lo < w.i_hi)
      for (int x = 0; x < heads; ++x) {
        cp_async_wait<W::kStages - 2>();
        __syncwarp();
        copy(stage == 0 ? W::kStages - 1 : stage - 1);
        uint32_t kf[2 * P][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < P; ++c) {
            uint4 v;
            const uint32_t at = mine + stage * W::kStage + (quad + 8 * r) * 2 * D + (((4 * c + kq) ^ quad) << 4);
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
            kf[2 * c][r] = v.x, kf[2 * c][r + 2] = v.y, kf[2 * c + 1][r] = v.z, kf[2 * c + 1][r + 2] = v.w;
          }
        tile_weights<T, D>(A, w, rs, hs + x * head_split, kf, acc, quad, kq);
        __syncwarp();
        stage = stage + 1 == W::kStages ? 0 : stage + 1;
      }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], 1);
      acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], 2);
    }
    if (kq == 0) {
      part[turn][warp][quad] = acc[0];
      part[turn][warp][quad + 8] = acc[1];
    }
    // a team's warps meet once a tile; two sets of sums keep a fast one from the next tile's
    if (head_split == 1)
      __syncwarp();
    else
      named_bar(1 + warp % teams, 32 * head_split);
    const int j = w.j0 + lane;
    if (warp < teams && lane < 16 && j < w.rq.n) {
      float sum = 0.f;
      for (int x = 0; x < head_split; ++x) sum += part[turn][warp + x * teams][lane];
      const int64_t at = w.b * A.score_stride + j;
      A.score_out[at] = (A.score_in ? A.decay * A.score_in[at] : 0.f) + sum;
    }
    turn ^= 1;
    if (head_split == 1) __syncwarp();
  }
  cp_async_wait<0>();
}

template <typename T, int D> static cudaError_t launch_weights_t(const PagedWeightsArgs &A, int split, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(paged_weights_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Weights<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_weights_kernel<T, D>, dim3(2 * num_sms()), dim3(32 * kWeightWarps), Weights<D>::kSmem, s, A, split);
}
static std::string launch_weights(const PagedWeightsArgs &A, int dtype, cudaStream_t s) {
  const PagedArgs &a = A.p;
  if (weights_many_takes(a)) return launch_weights_many(A, dtype, s);  // else pages make no boxes
  // Warps work on tiles of their own while there are enough for half of them; else they split the KV heads
  // of one (a token, 8 heads: 4096 slots 5.6 us split eight ways, 9.2 us whole; 16 384 slots 10.5 us
  // split in two, 12.2 us whole, 15.2 us split eight ways; 8 requests of 8192 slots 31.4 us whole, 34.7 us
  // split in two).
  int split = 1;
  const int64_t tiles = static_cast<int64_t>(a.n_requests) * ((a.max_len + 15) / 16), want = static_cast<int64_t>(kWeightWarps) * num_sms();
  while (split < kWeightWarps && 2 * split <= a.n_kv_heads && tiles * split < want) split *= 2;
  cudaError_t e;
  if (dtype == BD_BF16)
    e = a.head_dim == 128 ? launch_weights_t<__nv_bfloat16, 128>(A, split, s) : launch_weights_t<__nv_bfloat16, 64>(A, split, s);
  else
    e = a.head_dim == 128 ? launch_weights_t<__half, 128>(A, split, s) : launch_weights_t<__half, 64>(A, split, s);
  return e == cudaSuccess ? std::string() : std::string("paged weights: ") + cudaGetErrorString(e);
}

// ------------------------------------------------------------------ eviction
// Order-preserving integer image of a score: NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One cluster of blocks per request (one block up to kSelSmall slots, else eight).  Every warp has a run
// of slots of its own, in registers as far as they reach.  The key of the last slot that stays is found
// by radix selection, eleven, eleven and ten bits a pass: a histogram of the slots that match the bits
// found so far -- each block of its slots, summed over the cluster through distributed shared memory --
// then the digit that holds the wanted rank; it is done early where all slots of that digit stay.  Then each warp counts what stays of its run -- what is
// larger, and of what is equal the first ones -- and, knowing what stays before its run, places it.
// Bound by the round trips of its passes and barriers (a request of 4096 slots, 2048 kept: 11.3 us with
// the move).
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBlocks = 8;
constexpr int kSelSmall = 8192;
constexpr int kSelEach = 8;  // slots of a thread in registers
constexpr int kBins = 2048;

__device__ __forceinline__ int2 ld_cluster_i2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const __grid_constant__ PagedEvictArgs A) {
  __shared__ __align__(16) int hist[2][kBins];  // two: a block may clear one while others still read its last
  __shared__ int2 warp_cnt[kSelWarps];          // a run's slots that stay beside ties, and its ties
  __shared__ __align__(8) int2 block_cnt;
  __shared__ int warp_sum_s[kSelWarps];
  __shared__ uint32_t s_digit;
  __shared__ int2 s_need;  // slots wanted of the digit that holds the rank, and its slots
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const int blocks = gridDim.x, rank = blockIdx.x, ct = rank * kSelThreads + tid, CT = blocks * kSelThreads;  // of the cluster
  auto meet = [&]() {
    if (blocks > 1) cluster_sync(); else __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  const int n = request_len(A.p, b);
  const float *score = A.score + b * A.score_stride;
  float *score_out = A.score_out ? A.score_out + b * A.score_out_stride : nullptr;
  int32_t *kept = A.kept + static_cast<int64_t>(b) * A.budget;
  const bool in_place = score_out == score;
  if (n <= A.budget) {  // the whole cluster
    for (int j = ct; j < n; j += CT) {
      kept[j] = j;
      if (score_out && !in_place) score_out[j] = score[j];
    }
    meet();  // every thread has read the length: it may be replaced
    if (ct == 0) A.len_out[b] = n;
    return;
  }
  // slots [lo, hi) compete for `need` places; those outside stay
  const int lo = A.n_sink, hi = n - A.n_recent;
  int need = A.budget - A.n_sink - A.n_recent;
  const bool none = need == 0;
  // the warp's run: steps of 32 slots from j_lo on
  const int steps = (n + CT - 1) / CT, j_lo = (rank * kSelWarps + warp) * steps * 32 + lane;
  float held[kSelEach];
#pragma unroll
  for (int k = 0; k < kSelEach; ++k) held[k] = k < steps && j_lo + 32 * k < n ? score[j_lo + 32 * k] : 0.f;
  auto value = [&](int k, int j) { return j < n ? score[j] : 0.f; };  // beyond what is held
  uint32_t key = 0xffffffffu;  // key of the last one that stays (none: no score has this one)
  if (!none) {
    uint32_t mask = 0;
    key = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      int *h = hist[pass & 1];
      for (int d = tid; d < kBins; d += kSelThreads) h[d] = 0;
      __syncthreads();
      auto count = [&](int j, float v) {
        const uint32_t u = score_key(v);
        if (j >= lo && j < hi && (u & mask) == key) atomicAdd(&h[(u >> shift) & (bins - 1)], 1);
      };
#pragma unroll
      for (int k = 0; k < kSelEach; ++k)
        if (k < steps) count(j_lo + 32 * k, held[k]);
#pragma unroll 4
      for (int k = kSelEach; k < steps; ++k) count(j_lo + 32 * k, value(k, j_lo + 32 * k));
      meet();
      // thread t holds digits bins-1-2t and bins-2-2t, the larger first, of all blocks
      int c[2] = {0, 0};
      if (2 * tid < bins) {
        if (blocks == 1) {
          c[0] = h[bins - 1 - 2 * tid];
          c[1] = h[bins - 2 - 2 * tid];
        } else {
          const uint32_t at = smem_u32(h + bins - 2 - 2 * tid);
#pragma unroll
          for (int r = 0; r < kSelBlocks; ++r) {
            const int2 v = ld_cluster_i2(cluster_map(at, r));
            c[0] += v.y;
            c[1] += v.x;
          }
        }
      }
      int sum = c[0] + c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) warp_sum_s[warp] = sum;
      __syncthreads();
      int before = lane < warp ? warp_sum_s[lane] : 0;  // 32 warps: a lane each
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      before += sum - c[0] - c[1];
      if (before < need && before + c[0] + c[1] >= need) {
        const int x = before + c[0] < need;
        s_digit = bins - 1 - 2 * tid - x;
        s_need = make_int2(need - before - (x ? c[0] : 0), c[x]);
      }
      __syncthreads();
      key |= s_digit << shift;
      need = s_need.x;
      if (need == s_need.y && key > 0) {  // all of them stay: no need to tell them apart
        --key;
        need = 0;
        break;
      }
      mask |= (bins - 1u) << shift;
    }
  }
  // need: how many of the slots whose key is `key` stay (the first ones)
  int2 cnt = make_int2(0, 0);
  auto tally = [&](int j, float v) {
    const bool in = j >= lo && j < hi;
    const uint32_t u = score_key(v);
    cnt.x += __popc(__ballot_sync(0xffffffffu, j < n && (!in || u > key)));
    cnt.y += __popc(__ballot_sync(0xffffffffu, in && u == key));
  };
#pragma unroll
  for (int k = 0; k < kSelEach; ++k)
    if (k < steps) tally(j_lo + 32 * k, held[k]);
#pragma unroll 4
  for (int k = kSelEach; k < steps; ++k) tally(j_lo + 32 * k, value(k, j_lo + 32 * k));
  if (lane == 0) warp_cnt[warp] = cnt;
  __syncthreads();
  int2 at = lane < warp ? warp_cnt[lane] : make_int2(0, 0);
  if (blocks > 1) {
    if (warp == 0) {
      int2 all = warp_cnt[lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        all.x += __shfl_xor_sync(0xffffffffu, all.x, o);
        all.y += __shfl_xor_sync(0xffffffffu, all.y, o);
      }
      if (lane == 0) block_cnt = all;
    }
    cluster_sync();
    if (lane < rank) {  // the blocks before this one, a lane each
      const int2 v = ld_cluster_i2(cluster_map(smem_u32(&block_cnt), lane));
      at.x += v.x;
      at.y += v.y;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    at.x += __shfl_xor_sync(0xffffffffu, at.x, o);
    at.y += __shfl_xor_sync(0xffffffffu, at.y, o);
  }
  int larger = at.x, equal = at.y;  // before this run
  if (none) need = 0;
  auto place = [&](int j, float v) {
    const bool here = j < n, in = j >= lo && j < hi;
    const uint32_t u = score_key(v);
    const unsigned below = (1u << lane) - 1;
    const unsigned gt = __ballot_sync(0xffffffffu, here && (!in || u > key)), eq = __ballot_sync(0xffffffffu, in && u == key);
    const int e = equal + __popc(eq & below), to = larger + __popc(gt & below) + min(e, need);
    const bool keep = here && (!in || u > key || (u == key && e < need));
    larger += __popc(gt);
    equal += __popc(eq);
    if (keep) {
      kept[to] = j;
      if (score_out && !in_place) score_out[to] = v;
    }
  };
#pragma unroll
  for (int k = 0; k < kSelEach; ++k)
    if (k < steps) place(j_lo + 32 * k, held[k]);
#pragma unroll 1
  for (int k = kSelEach; k < steps; ++k) place(j_lo + 32 * k, value(k, j_lo + 32 * k));
  meet();  // kept[] is complete, every block's shared memory and the length are read
  if (in_place)
    // score i comes from kept[i] >= i: a step of them is written when all of it has been read, and the
    // steps behind it read behind what it wrote
    for (int i0 = 0; i0 < n; i0 += CT) {
      const int i = i0 + ct;
      const float v = i < A.budget ? __ldcg(score + __ldcg(kept + i)) : 0.f;
      meet();
      if (i < n) score_out[i] = v;  // behind the kept ones zero: slots filled later start from there
    }
  if (ct == 0) A.len_out[b] = A.budget;
}

// Moves the kept slots.  Slot i's row of one pool and KV head is D contiguous values; a thread moves 16
// bytes of it.  To other pages a block takes kMoveRows slots: it finds their places once, for `each` of
// the 2 Hkv row sets (pool and KV head), and has the next set's rows on the way while it writes one's.
// Bound by the bytes, read and written once (8 requests, up to 8192 slots kept: 101 us with the selection, 5.3 TB/s).
constexpr int kMoveThreads = 256;
constexpr int kMoveEach = 4;  // 16-byte pieces of a thread and row set

__device__ __forceinline__ int64_t dst_offset(const PagedEvictArgs &A, int b, int i) {
  if (!A.dst_table) return slot_offset(A.p, A.p.page_table + static_cast<int64_t>(b) * A.p.table_width, i);
  return slot_offset(A.p, A.dst_table + static_cast<int64_t>(b) * A.dst_width, i);
}

template <int CPR>  // pieces of a row
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const __grid_constant__ PagedEvictArgs A, int each) {
  const PagedArgs &a = A.p;
  const int b = blockIdx.z;
  pdl_wait();
  pdl_trigger();
  const int n = min(A.len_out[b], A.budget);
  constexpr int STEP = kMoveThreads / CPR, ROWS = STEP * kMoveEach;
  const int i0 = blockIdx.x * ROWS + threadIdx.x / CPR, x = (threadIdx.x % CPR) * 8;
  if (static_cast<int>(blockIdx.x) * ROWS >= n) return;
  const int32_t *kept = A.kept + static_cast<int64_t>(b) * A.budget;
  const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
  int j[kMoveEach];
#pragma unroll
  for (int u = 0; u < kMoveEach; ++u) j[u] = kept[min(i0 + u * STEP, n - 1)];
  int64_t src[kMoveEach], dst[kMoveEach];
#pragma unroll
  for (int u = 0; u < kMoveEach; ++u) {
    src[u] = slot_offset(a, table, j[u]);
    dst[u] = i0 + u * STEP < n ? dst_offset(A, b, i0 + u * STEP) : -1;
    if (src[u] < 0) dst[u] = -1;
  }
  const int s0 = blockIdx.y * each, s1 = min(2 * a.n_kv_heads, s0 + each);
  auto base = [&](int s) {
    return static_cast<uint16_t *>(const_cast<void *>(s & 1 ? a.v : a.k)) + (s >> 1) * a.head_stride + x;
  };
  uint4 v[kMoveEach];
  auto load = [&](int s) {
#pragma unroll
    for (int u = 0; u < kMoveEach; ++u)
      if (dst[u] >= 0) v[u] = __ldcs(reinterpret_cast<const uint4 *>(base(s) + src[u]));
  };
  load(s0);
  for (int s = s0; s < s1; ++s) {
    uint4 w[kMoveEach];
#pragma unroll
    for (int u = 0; u < kMoveEach; ++u) w[u] = v[u];
    if (s + 1 < s1) load(s + 1);
#pragma unroll
    for (int u = 0; u < kMoveEach; ++u)
      if (dst[u] >= 0) *reinterpret_cast<uint4 *>(base(s) + dst[u]) = w[u];
  }
}

// In place, one block per (request, KV head, pool) goes up through the slots in chunks of
// kChunkRows.  Slot i comes from old slot kept[i] >= i, so a chunk's writes can only hit rows that
// this chunk or an earlier one reads: a chunk is written after all of it has been read, and the
// next chunk's reads may go ahead of it.
constexpr int kInThreads = 512;
constexpr int kInRegs = 8;  // 16-byte pieces of a chunk per thread

__global__ void __launch_bounds__(kInThreads) paged_move_in_place_kernel(const __grid_constant__ PagedEvictArgs A) {
  const PagedArgs &a = A.p;
  const int b = blockIdx.y, h = blockIdx.x >> 1;
  if ((blockIdx.x & 1) && a.k == a.v) return;  // one pool for both: moved once, for two blocks would not keep in step
  uint16_t *pool = static_cast<uint16_t *>(const_cast<void *>(blockIdx.x & 1 ? a.v : a.k)) + h * a.head_stride;
  const int cpr = a.head_dim / 8;
  const int chunk = kInThreads * kInRegs / cpr;  // rows
  pdl_wait();
  pdl_trigger();
  const int n = min(A.len_out[b], A.budget);
  const int32_t *kept = A.kept + static_cast<int64_t>(b) * A.budget;
  const int32_t *table = a.page_table + static_cast<int64_t>(b) * a.table_width;
  for (int i0 = 0; i0 < n; i0 += chunk) {
    uint4 v[kInRegs];
    int64_t dst[kInRegs];
#pragma unroll
    for (int u = 0; u < kInRegs; ++u) {
      const int c = u * kInThreads + threadIdx.x, i = i0 + c / cpr, x = (c % cpr) * 8;
      dst[u] = -1;
      if (i < n) {
        const int j = kept[i];
        if (j != i) {
          const int64_t src = slot_offset(a, table, j), d = slot_offset(a, table, i);
          if (src >= 0 && d >= 0) {
            dst[u] = d + x;
            v[u] = *reinterpret_cast<const uint4 *>(pool + src + x);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kInRegs; ++u)
      if (dst[u] >= 0) *reinterpret_cast<uint4 *>(pool + dst[u]) = v[u];
  }
}

static std::string launch_evict(const PagedEvictArgs &A, cudaStream_t s) {
  const PagedArgs &a = A.p;
  // a barrier of eight blocks costs about a microsecond: fewer slots are one block's (a request of 4096
  // slots, 2048 kept: 16.3 us with eight blocks, 11.4 us with one; of 16 384: 16.0 and 18.8 us)
  const int sel = a.max_len <= kSelSmall ? 1 : kSelBlocks;
  cudaError_t e = launch_pdl_cluster(paged_select_kernel, dim3(sel, a.n_requests), dim3(kSelThreads), 0, s, sel, A);
  if (e == cudaSuccess) {
    const int most = A.budget < a.max_len ? A.budget : a.max_len;
    if (A.dst_table) {
      const int rows = kMoveThreads * kMoveEach / (a.head_dim / 8), blocks = (most + rows - 1) / rows, sets = 2 * a.n_kv_heads;
      // as many row sets a block as leave eight blocks an SM
      int each = 1;
      while (2 * each <= sets && static_cast<int64_t>(blocks) * a.n_requests * (sets / (2 * each)) >= 8 * num_sms()) each *= 2;
      const dim3 grid(blocks, (sets + each - 1) / each, a.n_requests);
      if (most > 0)
        e = launch_pdl(a.head_dim == 128 ? paged_move_kernel<16> : paged_move_kernel<8>, grid, dim3(kMoveThreads), 0, s, A, each);
    } else if (A.budget < a.max_len) {  // else nothing can leave
      e = launch_pdl(paged_move_in_place_kernel, dim3(2 * a.n_kv_heads, a.n_requests), dim3(kInThreads), 0, s, A);
    }
  }
  return e == cudaSuccess ? std::string() : std::string("paged eviction: ") + cudaGetErrorString(e);
}

// ------------------------------------------------------------------ host checks
namespace {

bd_status refuse(bd_status st, const std::string &msg) {
  set_last_error(msg);
  return st;
}
bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Whether [p, p + np) and [q, q + nq) (bytes) share any.
bool overlap(const void *p, int64_t np, const void *q, int64_t nq) {
  const char *a = static_cast<const char *>(p), *b = static_cast<const char *>(q);
  return np > 0 && nq > 0 && a < b + nq && b < a + np;
}

bd_status check_kv(const bd_paged_kv *c) {
  if (!c) return refuse(BD_ERR_INVALID_ARG, "paged kv is NULL");
  if (c->dtype != BD_BF16 && c->dtype != BD_F16)
    return refuse(BD_ERR_UNSUPPORTED, "paged kv: dtype must be BD_BF16 or BD_F16");
  if (c->head_dim != 64 && c->head_dim != 128) return refuse(BD_ERR_UNSUPPORTED, "paged kv: head_dim must be 64 or 128");
  if (c->n_kv_heads <= 0 || c->n_q_heads <= 0 || c->n_q_heads % c->n_kv_heads != 0)
    return refuse(BD_ERR_INVALID_ARG, "paged kv: n_q_heads must be a positive multiple of n_kv_heads");
  if (c->n_q_heads / c->n_kv_heads > BD_PAGED_MAX_GROUP || c->n_kv_heads > 1024)
    return refuse(BD_ERR_UNSUPPORTED, "paged kv: at most 128 query heads per KV head and 1024 KV heads");
  if (c->page_size < 1 || c->n_pages < 1) return refuse(BD_ERR_INVALID_ARG, "paged kv: page_size and n_pages must be >= 1");
  if (!c->k || !c->v || misaligned(c->k, 16) || misaligned(c->v, 16))
    return refuse(BD_ERR_INVALID_ARG, "paged kv: k and v must be 16-byte aligned pools");
  for (int64_t s : {c->page_stride, c->head_stride, c->slot_stride})
    if (s < 0 || s % 8) return refuse(BD_ERR_INVALID_ARG, "paged kv: strides must be multiples of 8 elements, >= 0");
  if ((c->page_size > 1 && c->slot_stride < c->head_dim) || (c->n_kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->n_pages > 1 && c->page_stride < c->head_dim))
    return refuse(BD_ERR_INVALID_ARG, "paged kv: strides must be at least head_dim elements");
  return BD_OK;
}

// Whether a slot's keys and values lie in one another but are not the same: no call can store them.
bool pools_mixed(const bd_paged_kv *c) { return c->k != c->v && overlap(c->k, 2 * c->head_dim, c->v, 2 * c->head_dim); }

bd_status check_batch(const bd_paged_kv *c, const bd_paged_batch *t, bool rows) {
  if (bd_status st = check_kv(c)) return st;
  if (!t) return refuse(BD_ERR_INVALID_ARG, "paged batch is NULL");
  if (t->n_requests < 1 || t->n_requests > BD_PAGED_MAX_REQUESTS)
    return refuse(BD_ERR_INVALID_ARG, "paged batch: n_requests must be in 1..1024");
  if (t->table_width < 1 || t->max_len < 0 ||
      t->max_len > static_cast<int64_t>(t->table_width) * c->page_size || t->max_len > (1 << 30))
    return refuse(BD_ERR_INVALID_ARG, "paged batch: max_len must be within table_width * page_size (and 2^30)");
  if (!t->page_table || !t->seq_len || misaligned(t->page_table, 4) || misaligned(t->seq_len, 4))
    return refuse(BD_ERR_INVALID_ARG, "paged batch: page_table and seq_len must be given");
  if (rows) {
    if (!t->row_start || misaligned(t->row_start, 4)) return refuse(BD_ERR_INVALID_ARG, "paged batch: row_start must be given");
    if (t->n_rows < 0 || t->max_rows < 0 || t->max_rows > t->n_rows || t->n_rows > (1 << 28))
      return refuse(BD_ERR_INVALID_ARG, "paged batch: 0 <= max_rows <= n_rows <= 2^28");
  }
  return BD_OK;
}

bd_status check_rows(const void *p, int64_t stride, int64_t width, int n_rows, const char *name) {
  if (!p || misaligned(p, 16) || stride % 8 || (n_rows > 1 && stride < width))
    return refuse(BD_ERR_INVALID_ARG, std::string("paged cache: ") + name +
                                          " must be 16-byte aligned rows with a stride that is a multiple of 8 and holds a row");
  return BD_OK;
}
int64_t row_bytes(int64_t stride, int64_t width, int n_rows) {
  return n_rows < 1 ? 0 : ((n_rows - 1) * stride + width) * 2;
}

bd_status check_mask(int window, int n_sink, float scale) {
  if (window < 0 || n_sink < 0) return refuse(BD_ERR_INVALID_ARG, "paged attention: window and n_sink must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale)) return refuse(BD_ERR_INVALID_ARG, "paged attention: scale must be > 0 and finite");
  return BD_OK;
}

PagedArgs args_of(const bd_paged_kv *c, const bd_paged_batch *t) {
  paged_used.store(true, std::memory_order_release);
  PagedArgs a = {};
  a.k = c->k;
  a.v = c->v;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  a.slot_stride = c->slot_stride;
  a.n_kv_heads = c->n_kv_heads;
  a.group = c->n_q_heads / c->n_kv_heads;
  a.head_dim = c->head_dim;
  a.page_size = c->page_size;
  a.n_pages = c->n_pages;
  a.n_requests = t->n_requests;
  a.table_width = t->table_width;
  a.n_rows = t->n_rows;
  a.max_rows = t->max_rows;
  a.max_len = t->max_len;
  a.page_table = t->page_table;
  a.seq_len = t->seq_len;
  a.row_start = t->row_start;
  return a;
}
bd_status ran(const std::string &e) { return e.empty() ? BD_OK : refuse(BD_ERR_CUDA, e); }

}  // namespace
}  // namespace bd

using namespace bd;

extern "C" {

size_t bd_paged_workspace_bytes(const bd_paged_kv *kv, int n_requests, int max_rows) {
  if (check_kv(kv)) return 0;
  if (n_requests < 1 || n_requests > BD_PAGED_MAX_REQUESTS || max_rows < 0) {
    refuse(BD_ERR_INVALID_ARG, "paged workspace: n_requests must be in 1..1024 and max_rows >= 0");
    return 0;
  }
  // a batch made for many rows may hold few (and the other way round): the larger of the two
  const size_t few = few_bytes(kv->head_dim);
  const size_t many = many_bytes(n_requests, max_rows, kv->n_q_heads / kv->n_kv_heads, kv->head_dim);
  return few > many ? few : many;
}

bd_status bd_paged_append(const bd_paged_kv *kv, const bd_paged_batch *batch, const void *k_new, int64_t k_stride,
                          const void *v_new, int64_t v_stride, void *stream) {
  if (bd_status st = check_batch(kv, batch, true)) return st;
  if (batch->n_rows == 0) return BD_OK;
  const int64_t width = static_cast<int64_t>(kv->n_kv_heads) * kv->head_dim;
  if (bd_status st = check_rows(k_new, k_stride, width, batch->n_rows, "k_new")) return st;
  if (bd_status st = check_rows(v_new, v_stride, width, batch->n_rows, "v_new")) return st;
  if (pools_mixed(kv) || (kv->k == kv->v && (k_new != v_new || k_stride != v_stride)))
    return refuse(BD_ERR_INVALID_ARG, "paged append: k and v are one pool, which takes the same rows as keys and values only");
  PagedAppendArgs A = {};
  A.p = args_of(kv, batch);
  A.k_new = k_new;
  A.v_new = v_new;
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  return ran(launch_append(A, static_cast<cudaStream_t>(stream)));
}

bd_status bd_paged_attention(const bd_paged_kv *kv, const bd_paged_batch *batch, const void *q, int64_t q_stride, void *out,
                             int64_t out_stride, float *lse, int window, int n_sink, float scale, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (bd_status st = check_batch(kv, batch, true)) return st;
  if (bd_status st = check_mask(window, n_sink, scale)) return st;
  if (batch->max_rows == 0) return BD_OK;
  const int64_t width = static_cast<int64_t>(kv->n_q_heads) * kv->head_dim;
  if (bd_status st = check_rows(q, q_stride, width, batch->n_rows, "q")) return st;
  if (bd_status st = check_rows(out, out_stride, width, batch->n_rows, "out")) return st;
  if (overlap(q, row_bytes(q_stride, width, batch->n_rows), out, row_bytes(out_stride, width, batch->n_rows)))
    return refuse(BD_ERR_INVALID_ARG, "paged attention: q and out overlap");
  if (misaligned(lse, 4)) return refuse(BD_ERR_INVALID_ARG, "paged attention: lse misaligned");
  if ((static_cast<int64_t>(batch->max_len) / 16 + 8) * kv->n_kv_heads >= (1ll << 31) ||
      static_cast<int64_t>(batch->max_rows) * kv->n_q_heads > (1 << 30) ||
      (static_cast<int64_t>(batch->max_rows) * (kv->n_q_heads / kv->n_kv_heads) / 256 + 1) * batch->n_requests > (1 << 28))
    return refuse(BD_ERR_UNSUPPORTED, "paged attention: max_len * n_kv_heads, max_rows * n_q_heads or n_requests * max_rows too large");
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < bd_paged_workspace_bytes(kv, batch->n_requests, batch->max_rows))
    return refuse(BD_ERR_WORKSPACE, "paged attention: workspace NULL, not 256-byte aligned or too small");
  PagedAttnArgs A = {};
  A.p = args_of(kv, batch);
  A.p.q = q;
  A.p.q_stride = q_stride;
  A.p.window = window;
  A.p.n_sink = n_sink;
  A.p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  A.out = out;
  A.out_stride = out_stride;
  A.lse = lse;
  const bool few = static_cast<int64_t>(batch->max_rows) * A.p.group <= kFewRows;
  return ran((few ? launch_attention_few : launch_attention_many)(A, workspace, kv->dtype, static_cast<cudaStream_t>(stream)));
}

bd_status bd_paged_weights(const bd_paged_kv *kv, const bd_paged_batch *batch, const void *q, int64_t q_stride,
                           const float *lse, const int32_t *rows_used, int window, int n_sink, float scale, float decay,
                           const float *score_in, float *score_out, int64_t score_stride, void *stream) {
  if (bd_status st = check_batch(kv, batch, true)) return st;
  if (bd_status st = check_mask(window, n_sink, scale)) return st;
  if (batch->max_len == 0) return BD_OK;
  const int64_t width = static_cast<int64_t>(kv->n_q_heads) * kv->head_dim;
  if (batch->max_rows > 0) {
    if (bd_status st = check_rows(q, q_stride, width, batch->n_rows, "q")) return st;
    if (!lse || misaligned(lse, 4)) return refuse(BD_ERR_INVALID_ARG, "paged weights: lse must be given");
  }
  if (misaligned(rows_used, 4)) return refuse(BD_ERR_INVALID_ARG, "paged weights: rows_used misaligned");
  if (static_cast<int64_t>(batch->max_rows) * kv->n_q_heads > (1 << 30) ||
      static_cast<int64_t>(batch->n_requests) * (batch->max_len / 16 + 1) >= (1ll << 30))
    return refuse(BD_ERR_UNSUPPORTED, "paged weights: max_rows * n_q_heads or n_requests * max_len too large");
  if (!std::isfinite(decay)) return refuse(BD_ERR_INVALID_ARG, "paged weights: decay must be finite");
  if (!score_out || misaligned(score_out, 4) || misaligned(score_in, 4) || score_stride < batch->max_len)
    return refuse(BD_ERR_INVALID_ARG, "paged weights: score_out must be given, with rows of at least max_len entries");
  const int64_t bytes = ((batch->n_requests - 1) * score_stride + batch->max_len) * 4;
  if (score_in && score_in != score_out && overlap(score_in, bytes, score_out, bytes))
    return refuse(BD_ERR_INVALID_ARG, "paged weights: score_in must be score_out or not overlap it");
  PagedWeightsArgs A = {};
  A.p = args_of(kv, batch);
  A.p.q = q;
  A.p.q_stride = q_stride;
  A.p.window = window;
  A.p.n_sink = n_sink;
  A.p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  A.lse = lse;
  A.rows_used = rows_used;
  A.decay = decay;
  A.score_in = score_in;
  A.score_out = score_out;
  A.score_stride = score_stride;
  return ran(launch_weights(A, kv->dtype, static_cast<cudaStream_t>(stream)));
}

bd_status bd_paged_evict(const bd_paged_kv *kv, const bd_paged_batch *batch, const float *score, int64_t score_stride,
                         int budget, int n_sink, int n_recent, const int32_t *dst_table, int dst_width, int32_t *kept_out,
                         int32_t *len_out, float *score_out, int64_t score_out_stride, void *stream) {
  if (bd_status st = check_batch(kv, batch, false)) return st;
  if (budget < 1 || n_sink < 0 || n_recent < 0 || static_cast<int64_t>(n_sink) + n_recent > budget)
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: budget must be >= 1 and hold n_sink + n_recent");
  if (pools_mixed(kv)) return refuse(BD_ERR_INVALID_ARG, "paged eviction: the slots of k and v overlap");
  const int most = budget < batch->max_len ? budget : batch->max_len;
  if (!score || misaligned(score, 4) || score_stride < batch->max_len)
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: score must be given, with rows of at least max_len entries");
  if (!kept_out || !len_out || misaligned(kept_out, 4) || misaligned(len_out, 4))
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: kept_out and len_out must be given");
  if (dst_table && (misaligned(dst_table, 4) || dst_width < 1 || static_cast<int64_t>(dst_width) * kv->page_size < most))
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: dst_table's rows must hold min(budget, max_len) slots");
  if (dst_table == batch->page_table && dst_table)
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: dst_table is page_table (NULL moves in place)");
  const int64_t ints = batch->n_requests * 4ll, kept = ints * budget, in = ((batch->n_requests - 1) * score_stride + batch->max_len) * 4;
  const int64_t out = score_out ? ((batch->n_requests - 1) * score_out_stride + most) * 4 : 0;
  if (score_out) {
    if (misaligned(score_out, 4) || score_out_stride < most)
      return refuse(BD_ERR_INVALID_ARG, "paged eviction: score_out's rows must hold min(budget, max_len) entries");
    if (score_out == score ? score_out_stride != score_stride : overlap(score, in, score_out, out))
      return refuse(BD_ERR_INVALID_ARG, "paged eviction: score_out must be score (same stride) or not overlap it");
  }
  if ((len_out != batch->seq_len && overlap(len_out, ints, batch->seq_len, ints)) || overlap(kept_out, kept, batch->seq_len, ints) ||
      overlap(kept_out, kept, len_out, ints) || overlap(kept_out, kept, score, in) || overlap(kept_out, kept, score_out, out) ||
      overlap(len_out, ints, score, in) || overlap(len_out, ints, score_out, out))
    return refuse(BD_ERR_INVALID_ARG, "paged eviction: kept_out, len_out (but for seq_len itself), seq_len, score and score_out overlap");
  PagedEvictArgs A = {};
  A.p = args_of(kv, batch);
  A.score = score;
  A.score_stride = score_stride;
  A.budget = budget;
  A.n_sink = n_sink;
  A.n_recent = n_recent;
  A.dst_table = dst_table;
  A.dst_width = dst_width;
  A.kept = kept_out;
  A.len_out = len_out;
  A.score_out = score_out;
  A.score_out_stride = score_out_stride;
  return ran(launch_evict(A, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
